"""The operators on a tree of drafted tokens at the edges of what their documentation allows.  Tolerances as in
test_draft_tree.py."""
import math

import pytest
import torch

import test_draft_tree as T
from test_attention_ops import ULP, assert_close, make_cache, offsets, ref_norm_rope, rotary_tables
from test_draft_tiles import FEW, TILED, TILES, kernel

from block_quantized_int8_q8_gb300 import api

gpu = pytest.mark.gpu
LOOSE = 1 << 20                                               # a loose bound of the lengths


# ------------------------------------------------------------------------------------------------ nothing to do
@gpu
def test_an_empty_batch_goes_through_every_operator():
    g = torch.Generator().manual_seed(1)
    cache, table = make_cache(g, [30, 40], 2, 64, 16, 16)
    before = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    rows = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    tb, kv, cu = table.cuda(), T.i32([30, 40]), T.i32([0, 0, 0])
    tree = api.draft_tree(T.i32([]), cu, 5)
    q = api.kv_append(cache, rows[:, 4:6], rows[:, 6:], tb, kv, cu, q=rows[:, :4], tree=tree)
    out, lse = api.attention(q, cache, tb, kv, 100, cu, 5, tree=tree, return_lse=True)
    assert q.shape == out.shape == (0, 4, 64) and lse.shape == (0, 4)
    api.kv_keep(cache, tb, kv, 0, T.i32([]).view(2, 0), T.i32([0, 0]), cu)
    assert api.read_device_errors() == 0
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


@gpu
def test_keep_of_no_rows():
    """No sequence keeps a token; a count that asks for one all the same is flagged."""
    g = torch.Generator().manual_seed(1)
    cache, table = make_cache(g, [30, 40], 2, 64, 16, 16)
    before = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    tb, kv, cu = table.cuda(), T.i32([30, 40]), T.i32([0, 6, 10])
    none = T.i32([]).view(2, 0)
    api.kv_keep(cache, tb, kv, 10, none, T.i32([0, 0]), cu)
    assert api.read_device_errors() == 0
    api.kv_keep(cache, tb, kv, 10, none, T.i32([0, 1]), cu)
    assert api.read_device_errors() == api.DEVERR_DRAFT
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


# ------------------------------------------------------------------------------------------------ tokens without a position
@gpu
@pytest.mark.parametrize("rot", [False, True])
@pytest.mark.parametrize("D,dt", [(64, torch.bfloat16), (128, torch.float32), (256, torch.float16)])
def test_append_writes_every_query_that_has_a_place(D, dt, rot):
    """A sequence shorter than its tokens (siblings turn at positions below 0, but have places) and depths below 0: without a
    rotation no position is needed; with one it is flagged and the row skipped."""
    g = torch.Generator().manual_seed(D)
    lens, n = [4, 20, 40], [6, 4, 3]
    cache, table = make_cache(g, lens, 2, D, 16, 16)
    tree = T.make_tree([[-1, 0, 0, 0, 0, 0], [-1, 0, 1, 0], [-1, -1, -1]], n)
    depths = tree.depths.clone()
    depths[7] = -20                                           # position -4
    depths[10] = -(2 ** 31)
    depths[11] = 2 ** 31 - 1
    tree = api.DraftTree(depths, tree.masks)
    first = [a - b for a, b in zip(lens, n)]
    seq = [i for i, k in enumerate(n) for _ in range(k)]
    place = [first[i] + j for i, k in enumerate(n) for j in range(k)]
    turn = [first[i] + int(d) for i, d in zip(seq, depths)]
    rows = torch.randn(sum(n), 8, D, generator=g).to(dt)
    dev = rows.cuda()
    w = 1 + 0.3 * torch.randn(D, generator=g)
    cos, sin = rotary_tables(64, D)
    q = torch.full((sum(n), 4, D), 9.0, device="cuda")
    api.read_device_errors()
    api.kv_append(cache, dev[:, 4:6], dev[:, 6:], table.cuda(), T.i32(lens), offsets(n).cuda(), cos.cuda() if rot else None,
                  sin.cuda() if rot else None, q=dev[:, :4], q_weight=w.cuda(), q_out=q, tree=tree)
    assert api.read_device_errors() == (api.DEVERR_LENGTH | (api.DEVERR_POSITION if rot else 0))
    k, _ = api.kv_read(cache, table.cuda(), T.i32([max(x, 0) for x in lens]), sum(lens), offsets(lens).cuda(), torch.float32)
    for t, (p, at) in enumerate(zip(place, turn)):
        if p < 0 or (rot and not 0 <= at < 64):
            assert (q[t] == 9).all(), t
            continue
        want = ref_norm_rope(rows[t, :4], w, 1e-6, *((cos[at], sin[at]) if rot else (None, None)), False)
        assert_close(q[t], want, 16 * 2.0 ** -24 * want.abs().amax(-1, keepdim=True) + 2.0 ** -24 * want.abs() + 1e-7, t)
        # its key is stored where its place says, to half a step of the block's scale
        got = k[int(offsets(lens)[seq[t]]) + p].cpu()
        key = ref_norm_rope(rows[t, 4:6], None, 1e-6, *((cos[at], sin[at]) if rot else (None, None)), False)
        step = cache.k_scale[int(table[seq[t], p // 16]), :, 0].double().cpu()[:, None]
        assert ((got.double() - key).abs() <= step * (0.5 + 2.0 ** -7) + 2.0 ** -20).all(), t


# ------------------------------------------------------------------------------------------------ depths that are no depths
@gpu
@pytest.mark.parametrize("depth", [0, 11, 12, 100, 100000, 2 ** 31 - 1, -1, -100, -(2 ** 31)])
@pytest.mark.parametrize("D,n,takes", [(64, 3, FEW), (64, 12, TILES), (64, 40, TILED), (128, 3, FEW), (128, 12, TILES),
                                       (128, 40, TILED), (256, 3, FEW), (256, 12, TILES), (256, 40, TILED)])
def test_window_takes_a_depth_past_the_bounds_as_the_nearest(D, n, takes, depth):
    """A depth that no tree of so many tokens has is flagged, and counts as the nearest that one has; every kernel agrees."""
    assert kernel(4, 2, D, 2, n, LOOSE) == takes
    g = torch.Generator().manual_seed(depth % 1000 + D)
    past, m, window = [900, 400], [n, 2], 200
    lens = [a + b for a, b in zip(past, m)]
    cache, table = make_cache(g, lens, 2, D, 64, 16)
    q = torch.randn(sum(m), 8, D, generator=g).bfloat16()
    parents = [T.draw_parents(k, g, "star") for k in m]
    tree = T.make_tree(parents, m)
    depths = tree.depths.clone()
    depths[1] = depth
    near = min(max(depth, 0), n - 1)
    api.read_device_errors()
    args = (q.cuda(), cache, table.cuda(), T.i32(lens), LOOSE, offsets(m).cuda(), n)
    out, lse = api.attention(*args, window=window, out_dtype=torch.float32, return_lse=True,
                             tree=api.DraftTree(depths, tree.masks))
    assert api.read_device_errors() == (api.DEVERR_DRAFT if near != depth else 0)
    want, wlse, vmax = T.ref_tree_attention(q, cache, table, lens, m, [T.sees(p) for p in parents], D ** -0.5, window)
    # the one row with another depth than its mask has
    first, ref = past[0], T.RefCache(cache)
    j = torch.arange(lens[0])
    see = torch.where(j < first, j > first + near - window, torch.cat([torch.zeros(first, dtype=torch.bool), T.sees(parents[0])[1]]))
    for h in range(8):
        k, v = (ref.values(side, table[0], 0, lens[0])[:, h // 4] for side in (0, 1))
        s = (k @ q[1, h].double() * D ** -0.5).masked_fill(~see, -math.inf)
        wlse[1, h], want[1, h] = torch.logsumexp(s, 0), torch.softmax(s, 0) @ v
    assert_close(out, want, torch.full_like(want, vmax * (2.0 ** -11 + 2.0 ** -16 + ULP[torch.float32])))
    assert ((lse.double().cpu() - wlse).abs() <= 2.0 ** -18 + 2.0 ** -20 * wlse.abs()).all()
    again = api.attention(*args, out_dtype=torch.float32, tree=api.DraftTree(depths, tree.masks))     # not looked at without a window
    assert torch.equal(again, api.attention(*args, out_dtype=torch.float32, tree=tree))
    assert api.read_device_errors() == 0


# ------------------------------------------------------------------------------------------------ rows of any magnitude
#: new tokens whose rows each kernel takes at four query heads for a key/value head under a loose bound, by head_dim
KERNELS = [(64, 3, FEW), (64, 12, TILES), (64, 30, TILES), (64, 40, TILED), (128, 3, FEW), (128, 12, TILES), (128, 30, TILES),
           (128, 40, TILED), (256, 3, FEW), (256, 12, TILES), (256, 40, TILED)]


@gpu
@pytest.mark.parametrize("small", [1.0, 2.0 ** -20])
@pytest.mark.parametrize("value", [3.0e38, -3.0e38, 1.0e30])
@pytest.mark.parametrize("D,n,takes", KERNELS)
def test_a_huge_finite_row_stays_alone(D, n, takes, value, small):
    """A finite row out of bounds, which no common factor with its neighbours may follow: they are what they are without it."""
    assert kernel(4, 2, D, 1, n, LOOSE) == takes
    g = torch.Generator().manual_seed(3)
    cache, table = make_cache(g, [300], 2, D, 64, 16)
    q = torch.randn(n, 8, D, generator=g).bfloat16() * small
    more = dict(scale=D ** -0.5 / small, out_dtype=torch.float32, return_lse=True, tree=T.make_tree([T.draw_parents(n, g)], [n]))
    args = (cache, table.cuda(), T.i32([300]), LOOSE, T.i32([0, n]), n)
    vmax = float((cache.v.abs().amax((2, 3)) * cache.v_scale.amax(-1)).max())
    want, wlse = api.attention(q.cuda(), *args, **more)
    x = q.clone()
    x[1, 3, 5] = value
    x[2, 6] = value
    got, lse = api.attention(x.cuda(), *args, **more)
    same = torch.ones(n, 8, dtype=torch.bool)
    same[1, 3] = same[2, 6] = False
    assert (got - want).abs()[same.cuda()].max() <= 2 * vmax * (2.0 ** -11 + 2.0 ** -16)
    assert ((lse - wlse).abs() <= 2.0 ** -17 + 2.0 ** -19 * wlse.abs())[same.cuda()].all()
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("D,n,takes", KERNELS)
def test_rows_of_many_magnitudes_over_tiny_scales(D, n, takes, monkeypatch):
    """Key scales of 2^-60: rows of 2^56 to 2^60 have ordinary scores, the others next to none, all within bounds."""
    assert kernel(4, 2, D, 2, n, LOOSE) == takes

    def tamper(cache, table, q):
        cache.k_scale.mul_(2.0 ** -60)
        q[0::3] *= 2.0 ** 60
        q[1::3] *= 2.0 ** 56
        q[2::3] *= 2.0 ** 30

    monkeypatch.setattr(T, "BOUND", LOOSE)
    T.check([300, 190], [n, 3], 8, 2, D, 64, 16, tamper=tamper)


# ------------------------------------------------------------------------------------------------ bounds that do not hold
@gpu
@pytest.mark.parametrize("bound", [200, 201, 128, 137])
@pytest.mark.parametrize("S,n,H,D,takes", [(1, 2, 2, 128, FEW), (256, 5, 8, 128, TILES), (256, 16, 16, 128, TILES),
                                           (128, 10, 32, 64, TILES), (60, 8, 16, 256, TILES), (2, 300, 8, 128, TILED)])
def test_tokens_past_the_stated_length_are_skipped(S, n, H, D, takes, bound):
    """Texts longer than the stated maximum are flagged, and no row sees a token past it."""
    assert kernel(4, H, D, S, n, bound) == takes
    g = torch.Generator().manual_seed(bound)
    length, few = 290 + n, min(S, 3)
    cache, table = make_cache(g, [length] * few, H, D, 64, 16)
    cache.v_scale[:, :, 0::4] *= 8.0                          # what comes after a boundary weighs
    q = torch.randn(few * n, 4 * H, D, generator=g).bfloat16()
    copies = [i % few for i in range(S)]
    rows = torch.cat([torch.arange(i * n, i * n + n) for i in copies])
    tree = T.make_tree([T.draw_parents(n, g)] * S, [n] * S)
    api.read_device_errors()
    out, lse = api.attention(q[rows].cuda(), cache, table[copies].cuda(), T.i32([length] * S), bound,
                             offsets([n] * S).cuda(), n, out_dtype=torch.float32, return_lse=True, tree=tree)
    assert api.read_device_errors() == api.DEVERR_LENGTH
    ref = T.RefCache(cache)
    want, wlse, vmax = torch.empty(few * n, 4 * H, D, dtype=torch.float64), torch.empty(few * n, 4 * H, dtype=torch.float64), 0.0
    for i in range(few):
        k, v = (ref.values(side, table[i], 0, bound) for side in (0, 1))
        vmax = max(vmax, float(v.abs().max()))
        for h in range(4 * H):
            s = q[i * n:i * n + n, h].double() @ k[:, h // 4].T * D ** -0.5
            wlse[i * n:i * n + n, h], want[i * n:i * n + n, h] = torch.logsumexp(s, -1), torch.softmax(s, -1) @ v[:, h // 4]
    assert_close(out, want[rows], torch.full_like(want[rows], vmax * (2.0 ** -11 + 2.0 ** -16 + ULP[torch.float32])))
    assert ((lse.double().cpu() - wlse[rows]).abs() <= 2.0 ** -18 + 2.0 ** -20 * wlse[rows].abs()).all()


# ------------------------------------------------------------------------------------------------ large caches
@gpu
@pytest.mark.parametrize("D,page,block", [(64, 16, 16), (128, 64, 16), (256, 64, 32)])
def test_caches_past_32_bits_of_bytes(D, page, block):
    """The same pages at the end of a cache of 4.3 GB of codes a side: every operator does what it does with them in a small one."""
    g = torch.Generator().manual_seed(D)
    H, n, lens = 2, [40, 3, 12], [700, 300, 1500]
    small, table = make_cache(g, lens, H, D, page, block)
    pages = (1 << 32) // (H * page * D) + 2 * small.pages
    big = api.KVCache(*(torch.empty((pages,) + x.shape[1:], dtype=x.dtype, device="cuda")
                        for x in (small.k, small.v, small.k_scale, small.v_scale)))
    shift = pages - small.pages
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(big, name)[shift:] = getattr(small, name)
    cu, kv, tree = offsets(n).cuda(), T.i32(lens), T.make_tree([T.draw_parents(k, g) for k in n], n)
    rows = torch.randn(sum(n), 8 + 2 * H, D, generator=g).bfloat16().cuda()
    cos, sin = (t.cuda() for t in rotary_tables(max(lens), D))
    got = []
    api.read_device_errors()
    for cache, tb in ((small, table), (big, torch.where(table >= 0, table + shift, table))):
        tb, out = tb.cuda(), []
        q = api.kv_append(cache, rows[:, 8:8 + H], rows[:, 8 + H:], tb, kv, cu, cos, sin, q=rows[:, :8], tree=tree)
        out.append(q)
        for some, takes in ((slice(0, 3), TILED), (slice(1, 3), TILES), (slice(1, 2), FEW)):
            at, m = slice(int(cu[some.start]), int(cu[some.stop])), max(n[some])
            assert kernel(4, H, D, len(n[some]), m, LOOSE) == takes
            out += api.attention(q[at], cache, tb[some].clone(), kv[some].clone(), LOOSE, cu[some.start:some.stop + 1] - cu[some.start],
                                 m, return_lse=True, tree=api.DraftTree(tree.depths[at].clone(), tree.masks[at].clone()))
        api.kv_keep(cache, tb, kv, sum(n), T.i32([[0, 5, 9, 31], [1, 2, 0, 0], [0, 1, 7, 11]]), T.i32([4, 2, 4]), cu)
        left = [a - b + c for a, b, c in zip(lens, n, (4, 2, 4))]
        out += api.kv_read(cache, tb, T.i32(left), sum(left), offsets(left).cuda(), torch.float32)
        got.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert api.read_device_errors() == 0
