"""Attention of a tree's rows in the kernel that shares out tiles (csrc/attn_tree.cu): every behaviour of the operator at sizes
that the rule of csrc/attn_api.cu sends there, which is asserted for each, and batches of which a block has more tiles than
it lists at once.  References and tolerances as in test_draft_tree.py."""
import ctypes
import math

import pytest
import torch

import test_draft_tree as T
from test_attention_ops import ULP, assert_close, make_cache, offsets

from block_quantized_int8_q8_gb300 import _build, api

gpu = pytest.mark.gpu
FEW, TILES, TILED = range(3)                                  # TreeKernel of csrc/attn.h
TILE, SHARES, LISTED = 128, 152, 256                          # tokens of a tile, blocks, tiles that a block lists at once
LOOSE = 1 << 20

#: rows (tokens x query heads of a group of 4) of the largest tree, for each head_dim
ROWS = [(64, 36), (64, 64), (64, 100), (64, 128), (128, 20), (128, 40), (128, 64), (128, 68), (128, 128), (256, 20), (256, 36),
        (256, 64)]


def kernel(group, kv_heads, dim, seqs, most, max_kv):
    _build.build()
    f = getattr(api.load(), "_ZN3mmq11tree_kernelEiiiixx")
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64] * 2
    f.restype = ctypes.c_int
    return f(group, kv_heads, dim, seqs, most, max_kv)


@pytest.fixture(autouse=True)
def loose(monkeypatch):
    """A loose bound of the lengths, with which short sequences take the kernel that long ones take."""
    monkeypatch.setattr(T, "BOUND", LOOSE)


def check(past, n, Hq, H, D, *args, **more):
    assert kernel(Hq // H, H, D, len(n), max(n), LOOSE) == TILES
    T.check(past, n, Hq, H, D, *args, **more)


@pytest.mark.parametrize("D,rows", ROWS)
def test_sizes_are_the_kernels(D, rows):
    for seqs in (1, 4, 700):
        assert kernel(4, 2, D, seqs, rows // 4, LOOSE) == TILES
    assert kernel(4, 2, D, 3, 1, LOOSE) == FEW and kernel(4, 2, D, 3, 33, LOOSE) == TILED


@gpu
@pytest.mark.parametrize("window", [1, 100, 128, 300, 5000])
@pytest.mark.parametrize("D,rows", ROWS)
def test_window(D, rows, window):
    n = rows // 4
    check([400, 150, 33, 2000, 129], [n, 3, n // 2, n, 1], 8, 2, D, 32, 16, window=max(window, n))


@gpu
@pytest.mark.parametrize("D,rows", ROWS)
def test_rows_without_a_place(D, rows):
    n = rows // 4
    check([-3, 5, -(n // 2), -n, -n - 9], [4, 3, n, n, n], 8, 2, D, 32, 16)
    check([-3, -1, -n // 2], [4, 1, n], 8, 2, D, 32, 16, kind="apart")
    check([-3, 200, -n // 2], [4, 1, n], 8, 2, D, 32, 16, window=n)


@gpu
@pytest.mark.parametrize("qt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ot", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,rows", [(64, 36), (64, 128), (128, 20), (128, 100), (256, 60)])
def test_types(qt, ot, D, rows):
    check([200, 77, 2500], [2, rows // 4, 3], 8, 2, D, 64, 32, qt, ot)


@gpu
@pytest.mark.parametrize("kind", ["forest", "path", "star", "apart"])
@pytest.mark.parametrize("D,rows", ROWS)
def test_kinds_of_trees(D, rows, kind):
    check([130, 0, 61, 1000], [rows // 8, 1, rows // 4, 3], 8, 2, D, kind=kind)


@gpu
@pytest.mark.parametrize("D,rows", ROWS)
def test_sharp_rows_and_scales(D, rows):
    def tamper(cache, table, q):
        q[0] *= 8.0
        cache.v_scale[int(table[0, 0]), :, 0] = 0
        cache.v[int(table[0, 0]), :, :16] = 0
        cache.v_scale[int(table[0, 2])] = 1e-7
        cache.k_scale[int(table[1, 0]), :, 0] = 0

    def tiny(cache, table, q):
        q *= 2.0 ** -100
        cache.v_scale.mul_(2.0 ** -30)

    n = [rows // 4, 3]
    check([300, 200], n, 8, 2, D, 64, 16, tamper=tamper)
    check([300, 200], n, 8, 2, D, 64, 16, tamper=tiny, scale=2.0 ** 97)
    check([300, 200], n, 8, 2, D, 64, 16, scale=-0.1)
    check([300, 200], n, 8, 2, D, 64, 16, scale=0.0)


@gpu
@pytest.mark.parametrize("D,rows", ROWS)
def test_reference_that_grows_late(D, rows):
    def tamper(cache, table, q):
        q.abs_()
        cache.k.copy_(torch.randint(60, 70, cache.k.shape, generator=torch.Generator().manual_seed(1)))
        for j, pg in enumerate(table[0].tolist()):
            if pg >= 0:
                cache.k_scale[pg] = 0.002 * (j + 1)
    check([1000], [rows // 4], 8, 2, D, 64, 16, tamper=tamper)
    check([1000], [rows // 4], 8, 2, D, 64, 16, tamper=tamper, scale=-D ** -0.5)


@gpu
@pytest.mark.parametrize("D,rows", ROWS)
def test_ignores_what_lies_past_the_length(D, rows):
    n = [rows // 8, rows // 4]
    assert kernel(4, 2, D, 2, max(n), LOOSE) == TILES
    T.test_attention_ignores_what_lies_past_the_length(n, D)


@gpu
@pytest.mark.parametrize("qt,ot", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
@pytest.mark.parametrize("D,rows", ROWS)
def test_strided_rows_streams_and_workspace(D, rows, qt, ot):
    """Queries and outputs that are slices of wider rows, another stream, a caller's workspace between two canaries; two runs: the
    same bits."""
    g = torch.Generator().manual_seed(11)
    n, lens = rows // 4, [3000, 2900]
    assert kernel(4, 2, D, 2, n, LOOSE) == TILES
    cache, table = make_cache(g, lens, 2, D, 64, 32)
    wide = torch.randn(2 * n, 13, D, generator=g).to(qt).cuda()
    q = wide[:, 2:10]
    tree = T.make_tree([T.draw_parents(n, g), T.draw_parents(n, g)], [n, n])
    kv, cu, tb = T.i32(lens), offsets([n, n]).cuda(), table.cuda()
    want, lse = api.attention(q.contiguous(), cache, tb, kv, LOOSE, cu, n, tree=tree, out_dtype=ot, return_lse=True)
    need = api.attention_tree_workspace_bytes(2 * n, 8, 2, D, 2, n, LOOSE)
    ws = torch.full((64 + need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((2 * n + 2, 12, D), 5.0, dtype=ot, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _, again = api.attention(q, cache, tb, kv, LOOSE, cu, n, out=out[1:-1, 1:9], workspace=ws[64:64 + need], stream=st, tree=tree,
                             return_lse=True)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out[1:-1, 1:9], want) and torch.equal(lse, again)
    assert (out[:, 0] == 5).all() and (out[:, 9:] == 5).all() and (out[0] == 5).all() and (out[-1] == 5).all()
    assert (ws[:64] == 0xFF).all() and (ws[64 + need:] == 0xFF).all()


@gpu
@pytest.mark.parametrize("D,rows", ROWS)
def test_a_path_is_causal_attention(D, rows):
    g = torch.Generator().manual_seed(8)
    n, lens = [rows // 8, rows // 4, 1], [800, rows // 4, 400]
    assert kernel(4, 2, D, 3, max(n), LOOSE) == TILES
    cache, table = make_cache(g, lens, 2, D, 64, 16)
    q = torch.randn(sum(n), 8, D, generator=g).bfloat16().cuda()
    args = (q, cache, table.cuda(), T.i32(lens), LOOSE, offsets(n).cuda(), max(n))
    more = dict(out_dtype=torch.float32, return_lse=True)
    a, la = api.attention(*args, **more)
    b, lb = api.attention(*args, **more, tree=T.make_tree([T.draw_parents(k, g, "path") for k in n], n))
    vmax = float((cache.v.abs().amax((2, 3)) * cache.v_scale.amax(-1)).max())
    assert (a - b).abs().max() <= vmax * 2 * (2.0 ** -11 + 2.0 ** -16) and (la - lb).abs().max() <= 2.0 ** -17 + 2.0 ** -19 * 12


# ------------------------------------------------------------------------------------------------ more than one list of tiles
def pool_cache(g, pages, H, D):
    """A cache of few pages of 64 tokens, which tables name again and again."""
    def side():
        return (torch.randn(pages, H, 64, D, generator=g) * 40).round().clamp(-127, 127).to(torch.int8).cuda()

    return api.KVCache(side(), side(), *((torch.rand(pages, H, 4, generator=g) * 0.02 + 0.01).cuda() for _ in range(2)))


def reference(q, masks, cache, row, length, window):
    """out and lse of one sequence's n rows in 64 bits; masks bool [n, n]."""
    n, Hq, D = q.shape
    group, first = Hq // cache.kv_heads, length - q.shape[0]
    at = torch.arange(length, device="cuda")
    page, off = row[at // cache.page_size].long(), at % cache.page_size
    see = torch.ones(n, length, dtype=torch.bool, device="cuda")
    see[:, first:] = masks.cuda()
    if window:
        place = first + masks.sum(-1, keepdim=True).cuda() - 1
        see &= (at > place - window) | (at >= first)
    out = torch.empty(n, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(n, Hq, dtype=torch.float64, device="cuda")
    for h in range(cache.kv_heads):
        k, v = (c[page, h, off].double() * s[page, h, off // cache.block].double()[:, None]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        s = (q[:, h * group:(h + 1) * group].double() @ k.T * D ** -0.5).masked_fill(~see[:, None], -math.inf)
        lse[:, h * group:(h + 1) * group] = torch.logsumexp(s, -1)
        out[:, h * group:(h + 1) * group] = torch.softmax(s, -1) @ v
    return out.cpu(), lse.cpu()


@gpu
@pytest.mark.parametrize("D,Hq,most,seqs,window,texts", [
    # up to 256 (R = 128: 512) sequences fit the first look at the batch; of the texts, what a window leaves counts
    (64, 64, 8, 240, 0, [2, 127, 4000, 6001, 9000, 131072]),
    (128, 32, 9, 900, 0, [0, 120, 1500, 2048, 3333, 131072]),
    (128, 32, 30, 430, 0, [31, 129, 2500, 4096, 5555, 120001]),
    (128, 32, 16, 800, 3000, [0, 100, 2984, 4000, 5000, 20000]),
    (256, 32, 12, 350, 0, [5, 700, 3000, 4999, 8000, 120000]),
])
def test_blocks_list_their_tiles_more_than_twice(D, Hq, most, seqs, window, texts):
    """Shares of more than two lists: units that go on in the next list, that end one, that lie across blocks and lists both; the
    sequences are copies of a few, whose results are known."""
    H, P = 8, 64
    g = torch.Generator().manual_seed(seqs + D)
    pool = 53
    cache = pool_cache(g, pool, H, D)
    n = [most, 1, most - 1, most, most // 2, most - 2]
    lens = [a + b for a, b in zip(texts, n)]
    parents = [T.draw_parents(k, g) for k in n]
    masks = [T.sees(p) for p in parents]
    tables = [torch.randint(0, pool, (-(-max(lens) // P),), generator=g, dtype=torch.int32) for _ in n]
    q = [torch.randn(k, Hq, D, generator=g).bfloat16() for k in n]
    # a few of the longest, the others of every other length; some sequences without new tokens
    order = [5 if i in (3, seqs // 2, seqs - 2) else (-1 if i % 41 == 7 else int(torch.randint(0, 5, (1,), generator=g)))
             for i in range(seqs)]
    tiles = [-(-(b - max(a - window + 1, 0) // 16 * 16 if window else b) // TILE) for a, b in zip(texts, lens)]
    total = H * sum(tiles[k] for k in order if k >= 0)
    assert total > 2 * SHARES * LISTED, total
    if not window:
        assert tiles[5] > LISTED + total // SHARES            # across two blocks, and two lists of the first
    assert kernel(Hq // H, H, D, seqs, most, max(lens)) == TILES
    kv_lens = [lens[k] if k >= 0 else 500 for k in order]
    new = [n[k] if k >= 0 else 0 for k in order]
    tree = T.make_tree([parents[k] if k >= 0 else [] for k in order], new)
    api.read_device_errors()
    out, lse = api.attention(torch.cat([q[k] for k in order if k >= 0]).cuda(), cache,
                             torch.stack([tables[max(k, 0)] for k in order]).cuda(), T.i32(kv_lens), max_kv_len=max(lens),
                             cu_tokens=offsets(new).cuda(), max_tokens=most, window=window, out_dtype=torch.float32,
                             return_lse=True, tree=tree)
    assert api.read_device_errors() == 0
    vmax = float((cache.v.abs().amax((2, 3)) * cache.v_scale.amax(-1)).max())
    wants = [reference(x.cuda(), m, cache, t.cuda(), L, window) for x, m, t, L in zip(q, masks, tables, lens)]
    out, lse, at = out.cpu(), lse.cpu(), offsets(new).tolist()
    for i, k in enumerate(order):
        if k < 0:
            continue
        want, wlse = wants[k]
        assert_close(out[at[i]:at[i + 1]], want, torch.full_like(want, vmax * (2.0 ** -11 + 2.0 ** -16 + ULP[torch.float32])),
                     f"sequence {i} of kind {k}")
        assert ((lse[at[i]:at[i + 1]].double() - wlse).abs() <= 2.0 ** -18 + 2.0 ** -20 * wlse.abs()).all(), (i, k)


@gpu
@pytest.mark.parametrize("D,Hq,H,n,seqs", [(64, 64, 8, 8, 16), (64, 32, 8, 10, 40), (128, 32, 8, 9, 24), (128, 32, 8, 30, 16),
                                           (256, 16, 4, 12, 32)])
def test_calls_repeat_to_the_bit(D, Hq, H, n, seqs):
    """Ragged texts of up to 8192 tokens, the same call again and again: a result that is read before its last product is there
    differs from one call to the next."""
    g = torch.Generator().manual_seed(seqs + D)
    cache = pool_cache(g, 300, H, D)
    lens = (torch.rand(seqs, generator=g) * 8192).int().tolist()
    lens = [x + n for x in lens]
    table = torch.randint(0, 300, (seqs, -(-max(lens) // 64)), generator=g, dtype=torch.int32)
    assert kernel(Hq // H, H, D, seqs, n, max(lens)) == TILES
    parents = [T.draw_parents(n, g) for _ in lens]
    q = torch.randn(seqs * n, Hq, D, generator=g).bfloat16()
    tree, args = T.make_tree(parents, [n] * seqs), (q.cuda(), cache, table.cuda(), T.i32(lens), max(lens), offsets([n] * seqs).cuda(), n)
    first = [x.clone() for x in api.attention(*args, tree=tree, return_lse=True, out_dtype=torch.float32)]
    for _ in range(20):
        again = api.attention(*args, tree=tree, return_lse=True, out_dtype=torch.float32)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    vmax = float((cache.v.abs().amax((2, 3)) * cache.v_scale.amax(-1)).max())
    for i in (0, seqs // 2, seqs - 1):
        at = slice(i * n, i * n + n)
        want, _ = reference(q[at].cuda(), T.sees(parents[i]), cache, table[i].cuda(), lens[i], 0)
        assert_close(first[0][at], want, torch.full_like(want, vmax * (2.0 ** -11 + 2.0 ** -16 + ULP[torch.float32])))
    assert api.read_device_errors() == 0
