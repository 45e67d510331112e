"""The operators on a tree of drafted tokens at the edges of what their documentation allows.  Tolerances as in
test_draft_tree.py."""
import pytest
import torch

import test_draft_tree as T
from test_attention_ops import assert_close, make_cache, offsets, ref_norm_rope, rotary_tables

from block_quantized_int8_q8_gb300 import api

gpu = pytest.mark.gpu


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
