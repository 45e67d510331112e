"""Host-side checks of the boundary of the operators on a tree of drafted tokens (no GPU needed).  Arguments are refused before
any CUDA call, so the pointers here are fake and never dereferenced."""
import struct

import pytest

from test_attention_host import (ALIGN, CACHE_AND_SEQS, F16, F32, FAKE, INVALID, SHAPE, UNSUPPORTED, cache, heads, lib,
                                 rotary, seqs)  # noqa: F401

from block_quantized_int8_q8_gb300 import api

TREE = struct.Struct("@PPi4x")                                # depths, masks, mask_words


def tree(depths=FAKE, masks=FAKE, words=1):
    return TREE.pack(depths or 0, masks or 0, words)


@pytest.mark.parametrize("kw,status", [
    (dict(parents=None), INVALID),
    (dict(depths=None), INVALID),
    (dict(masks=None), INVALID),
    (dict(seqs=-1), INVALID),
    (dict(seqs=0), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(max_tokens=-1), INVALID),
    (dict(max_tokens=0), INVALID),
    (dict(words=-1), INVALID),
    (dict(cu=None), INVALID),                                 # five tokens, three sequences
    (dict(max_tokens=1025, words=64), SHAPE),
    (dict(max_tokens=33), SHAPE),                             # more than the words hold
    (dict(tokens=1 << 31), SHAPE),
    (dict(tokens=1 << 30, words=4), SHAPE),
    (dict(parents=FAKE + 4), ALIGN),
    (dict(cu=FAKE + 8), ALIGN),
    (dict(depths=FAKE + 4), ALIGN),
    (dict(masks=FAKE + 4), ALIGN),
    (dict(tokens=0, parents=None, depths=None, masks=None), 0),
    (dict(tokens=0, seqs=0), 0),
])
def test_masks_refusals(lib, kw, status):  # noqa: F811
    a = dict(parents=FAKE, cu=FAKE, seqs=3, tokens=5, max_tokens=4, depths=FAKE, masks=FAKE, words=1)
    a.update(kw)
    assert lib.mmq_draft_masks(a["parents"], a["cu"], a["seqs"], a["tokens"], a["max_tokens"], a["depths"], a["masks"],
                               a["words"], None) == status


@pytest.mark.parametrize("kw,status", CACHE_AND_SEQS + [
    (dict(t=None), INVALID),
    (dict(t=tree(depths=None)), INVALID),
    (dict(t=tree(depths=FAKE + 4)), ALIGN),
    (dict(k=None), INVALID),
    (dict(v=heads(dtype=F32)), UNSUPPORTED),
    (dict(q=heads(), qo=None, hq=4), INVALID),
    (dict(q=heads(dtype=F16), qo=heads(), hq=4), UNSUPPORTED),
    (dict(rot=rotary(rot=256)), SHAPE),
    (dict(t=tree(masks=None, words=0), tokens=0), 0),
])
def test_append_refusals(lib, kw, status):  # noqa: F811
    a = dict(c=cache(), s=seqs(), t=tree(masks=None), tokens=5, k=heads(), v=heads(), q=None, hq=0, qo=None, rot=None)
    a.update(kw)
    assert lib.mmq_kv_append_tree(a["c"], a["s"], a["t"], a["tokens"], a["k"], a["v"], None, a["q"], a["hq"], None, a["qo"],
                                  a["rot"], 1e-6, None) == status


@pytest.mark.parametrize("kw,status", CACHE_AND_SEQS + [
    (dict(kept=None), INVALID),
    (dict(counts=None), INVALID),
    (dict(stride=-1), INVALID),
    (dict(stride=1025), SHAPE),
    (dict(kept=FAKE + 4), ALIGN),
    (dict(counts=FAKE + 4), ALIGN),
])
def test_keep_refusals(lib, kw, status):  # noqa: F811
    a = dict(c=cache(), s=seqs(), tokens=5, kept=FAKE, stride=4, counts=FAKE)
    a.update(kw)
    assert lib.mmq_kv_keep(a["c"], a["s"], a["tokens"], a["kept"], a["stride"], a["counts"], None) == status


def test_binding_refuses_what_it_cannot_pass(lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: api.draft_tree(x), lambda: api.draft_tree(x.float()), lambda: api.draft_tree(x[None]),
                 lambda: api.draft_tree(None), lambda: api._of_tree((x, x)), lambda: api._of_tree(x)):
        with pytest.raises(api.MMQError):
            call()
