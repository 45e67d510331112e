"""Host-side checks of the boundary of the operators on a tree of drafted tokens (no GPU needed).  Arguments are refused before
any CUDA call, so the pointers here are fake and never dereferenced."""
import ctypes
import random
import struct

import pytest

from test_attention_host import (ALIGN, BF16, CACHE_AND_SEQS, F16, F32, FAKE, INVALID, SHAPE, UNSUPPORTED, WORKSPACE, cache,
                                 heads, lib, rotary, seqs)  # noqa: F401

from test_attention_plan import Plan, device_parts

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
    (dict(t=None), INVALID),
    (dict(t=tree(masks=None)), INVALID),
    (dict(t=tree(depths=None), window=500), INVALID),         # a window goes by depth
    (dict(t=tree(masks=FAKE + 4)), ALIGN),
    (dict(t=tree(depths=FAKE + 4)), ALIGN),
    (dict(t=tree(words=0)), SHAPE),
    (dict(t=tree(words=1 << 30)), SHAPE),
    (dict(tokens=2000, max_tokens=1025, t=tree(words=33)), SHAPE),
    (dict(tokens=40, max_tokens=33), SHAPE),                  # more tokens than a mask's words hold
    (dict(window=3, max_tokens=4), UNSUPPORTED),              # could hide a drafted token
    (dict(window=-1), INVALID),
    (dict(hq=0), INVALID),
    (dict(hq=7), SHAPE),
    (dict(tokens=1 << 30), SHAPE),
    (dict(max_tokens=0), INVALID),
    (dict(max_tokens=-1), INVALID),
    (dict(max_kv=-1), INVALID),
    (dict(max_kv=1 << 31), SHAPE),
    (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(q=heads(dtype=F32)), UNSUPPORTED),
    (dict(q=heads(data=None)), INVALID),
    (dict(out=None), INVALID),
    (dict(out=heads(ts=4)), ALIGN),
    (dict(lse=FAKE + 4), ALIGN),
    (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=-1), WORKSPACE),                           # one byte short
    (dict(ws=FAKE + 8), ALIGN),
])
def test_attention_refusals(lib, kw, status):  # noqa: F811
    a = dict(c=cache(), s=seqs(), t=tree(), tokens=5, hq=4, q=heads(), out=heads(), max_tokens=4, max_kv=100000, scale=0.1,
             window=0, lse=None, ws=FAKE, ws_bytes=0)
    a.update(kw)
    need = lib.mmq_attention_tree_workspace_bytes(5, 4, 2, 128, 3, 4, 100000)
    assert need > 0
    assert lib.mmq_attention_tree(a["q"], a["hq"], a["c"], a["s"], a["t"], a["tokens"], a["max_tokens"], a["max_kv"],
                                  a["scale"], a["window"], a["out"], a["lse"], a["ws"], need + a["ws_bytes"],
                                  None) == status


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


def test_workspace_sizes(lib):  # noqa: F811
    size = lib.mmq_attention_tree_workspace_bytes
    assert size(26, 32, 8, 128, 1, 26, 100000) >= 26 * 32 * 128 * 4
    for bad in ((0, 32, 8, 128, 1, 26, 1000), (26, 32, 7, 128, 1, 26, 1000), (26, 32, 8, 96, 1, 26, 1000),
                (26, 32, 8, 128, 0, 26, 1000), (26, 32, 8, 128, 1, 0, 1000), (26, 32, 8, 128, 1, 26, -1),
                (2000, 32, 8, 128, 1, 1025, 1000)):
        assert size(*bad) == 0, bad


def test_line_of_tiles_is_bounded(lib):  # noqa: F811
    """What the kernel numbers with 32 bits: the bounds' tiles over all sequences and heads."""
    size = lib.mmq_attention_tree_workspace_bytes
    big, most = 1 << 20, ((1 << 30) // (16 * 8192) - 6) * 128
    for tokens, kv_heads, n, max_kv, fits in ((8192, 16, 8192, most - 128, True), (8192, 16, 8192, most, False),
                                                 (big, 64, big, 100000, False)):
        assert (size(tokens, kv_heads, kv_heads, 128, n, 32, max_kv) > 0) == fits
        if not fits:
            assert lib.mmq_attention_tree(heads(), kv_heads, cache(h=kv_heads), seqs(n=n), tree(), tokens, 32, max_kv, 0.1, 0,
                                          heads(), None, FAKE, 1 << 40, None) == SHAPE


def test_parts_of_a_tree_fit_the_launch_and_the_workspace(lib):  # noqa: F811
    """As test_attention_plan.py has it, for a tree's rows: many in the few-row kernel, few in the kernel of prompts."""
    plan = getattr(lib, "_ZN3mmq17attention_plan_ofEbxiiiixxx")
    plan.argtypes = [ctypes.c_bool, ctypes.c_int64] + [ctypes.c_int] * 4 + [ctypes.c_int64] * 3
    plan.restype = Plan
    rng = random.Random(4)
    for _ in range(4000):
        kv, dim, few = rng.choice([1, 2, 8]), rng.choice([64, 128, 256]), rng.random() < 0.5
        heads, seqs = kv * rng.choice([1, 3, 4, 8, 32]), int(2 ** rng.uniform(0, 9))
        most, max_kv = int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 18))
        tokens = rng.randint(max(most, seqs), max(seqs * most, most, seqs))
        window = rng.choice([0, 0, most, most + 16, max_kv // 2, max_kv, (1 << 63) - 1])
        p, whole = (plan(few, tokens, heads, kv, dim, seqs, most, max_kv, w) for w in (window, 0))
        assert p.few == few and p.total <= whole.total and p.chunk > 0 and p.chunk % 16 == 0
        assert p.chunk <= 2048 if few else (p.total > 0) == (p.splits > 1 or p.chunk > 32768)
        assert p.total > 0 or p.splits == 1
        if p.total > 0:
            rows = tokens * heads * p.splits
            assert p.part_o >= rows * 8 and p.total - p.part_o >= rows * dim * 4
        for length in {0, 1, max_kv - 1, max_kv, max_kv + 7, rng.randint(0, max_kv)}:
            for n in {1, most, most + 3, rng.randint(1, most)}:
                assert device_parts(max(length, 0), n, p.chunk, True, p.window, most, max_kv) <= p.splits


def test_binding_refuses_what_it_cannot_pass(lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: api.draft_tree(x), lambda: api.draft_tree(x.float()), lambda: api.draft_tree(x[None]),
                 lambda: api.draft_tree(None), lambda: api._of_tree((x, x)), lambda: api._of_tree(x)):
        with pytest.raises(api.MMQError):
            call()
