"""Host-side checks of the operators on a tree of drafted tokens where there is nothing to do, and of the binding's tree object
(no GPU needed).  The pointers are fake and never dereferenced."""
import pytest

from test_attention_host import FAKE, INVALID, cache, heads, lib, seqs  # noqa: F401
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
