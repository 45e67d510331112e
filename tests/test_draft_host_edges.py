"""Host-side checks of the operators on a tree of drafted tokens where there is nothing to do, and of the binding's tree object
(no GPU needed).  The pointers are fake and never dereferenced."""
import pytest

from block_quantized_int8_q8_gb300 import api
from test_attention_host import ALIGN, FAKE, INVALID, cache, heads, lib, seqs  # noqa: F401
from test_draft_host import tree


@pytest.mark.parametrize("t,tokens,status", [
    (tree(depths=None, masks=None, words=0), 0, 0),           # an empty tensor's pointer is null
    (tree(depths=FAKE + 4), 0, 0),
    (tree(depths=None), 5, INVALID),
    (None, 0, INVALID),
])
def test_append_of_no_tokens_needs_no_depths(lib, t, tokens, status):  # noqa: F811
    assert lib.mmq_kv_append_tree(cache(), seqs(), t, tokens, heads(), heads(), None, None, 0, None, None, None, 1e-6,
                                  None) == status


@pytest.mark.parametrize("kept,stride,counts,tokens,status", [
    (None, 0, None, 5, INVALID),
    (None, 4, FAKE, 5, INVALID),
    (None, 0, FAKE, 0, 0),
    (FAKE + 4, 0, FAKE, 5, ALIGN),
])
def test_keep_refuses_rows_that_are_not_there(lib, kept, stride, counts, tokens, status):  # noqa: F811
    assert lib.mmq_kv_keep(cache(), seqs(), tokens, kept, stride, counts, None) == status


def test_keep_of_no_rows_needs_none(lib):  # noqa: F811
    """A null array of no rows gets past the checks: the next one, of the counts' alignment, is what refuses the call."""
    assert lib.mmq_kv_keep(cache(), seqs(), 5, None, 0, FAKE + 4, None) == ALIGN
    assert lib.mmq_kv_keep(cache(), seqs(), 5, None, 1, FAKE + 4, None) == INVALID


def test_a_tree_without_its_tensors_is_not_no_tree(lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, dtype=torch.int32)
    for t in (api.DraftTree(None, None), api.DraftTree(x, None), api.DraftTree(None, x[:, None])):
        with pytest.raises(api.MMQError):
            api._of_tree(t)
    assert api._of_tree(None) == (None, None)
    t = api.DraftTree(x, x[:, None])
    assert api._of_tree(t)[0] is t.depths and api._of_tree(t)[1] is t.masks
