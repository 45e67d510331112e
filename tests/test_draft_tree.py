"""The operators that check a tree of drafted tokens over the 8-bit paged cache, against plain implementations.

Tolerances:
  masks, keep  whole numbers and f32 quotients of two f32 numbers: equal to the bit.
  append       as in test_attention_ops.py (the same arithmetic, other positions), the reference's quotients and product of
               the rescale in f32, as they are defined: fp16 and bf16 rows hold exact halves of a code, where 64 bits and
               the definition part.
  attention    as in test_attention_ops.py: probabilities as fp16, half a step of 2^-11 each, over values of magnitude
               <= vmax, 2^-16 of vmax for queries and scores, half a step of the output type; lse 2^-18 + 2^-20 |lse|.
"""
import math
import sys

import pytest
import torch

from test_attention_sizes import ExactCache
from test_attention_ops import (RefCache, ULP, assert_cache, assert_close, make_cache, offsets, ref_norm_rope,
                                rotary_tables)

from block_quantized_int8_q8_gb300 import api

gpu = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def draw_parents(n, g, kind="any"):
    """Parents of one sequence's n tokens: a path, a star, one tree or several."""
    if kind == "path":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    if kind == "apart":
        return [-1] * n
    u = torch.rand(n, 2, generator=g)
    low = -1 if kind == "forest" else 0
    return [-1 if i == 0 else (i - 1 if u[i, 0] < 0.3 else low + int(u[i, 1] * (i - low))) for i in range(n)]


def sees(parents):
    """Row i sees column j, in the plain way."""
    m = torch.zeros(len(parents), len(parents), dtype=torch.bool)
    for i, p in enumerate(parents):
        m[i, i] = True
        while p >= 0:
            m[i, p] = True
            p = parents[p]
    return m


def make_tree(parents, n):
    """DraftTree of the sequences' parents, made on the CPU."""
    words = max(1, -(-max(n) // 32))
    masks = torch.zeros(sum(n), words * 32, dtype=torch.int64)
    depths, at = [], 0
    for p in parents:
        m = sees(p)
        masks[at:at + len(p), :len(p)] = m.long()
        depths += (m.sum(-1) - 1).tolist()
        at += len(p)
    packed = (masks.view(sum(n), words, 32) << torch.arange(32)).sum(-1).to(torch.int32)
    return api.DraftTree(i32(depths), packed.cuda())


# ------------------------------------------------------------------------------------------------ masks
@gpu
@pytest.mark.parametrize("kind", ["any", "forest", "path", "star", "apart"])
@pytest.mark.parametrize("n", [[1], [26], [33, 0, 1, 32, 64], [5, 31, 65, 128, 127], [300, 2, 257], [1024, 1023, 7],
                               [3] * 700])
def test_masks(kind, n):
    g = torch.Generator().manual_seed(sum(n))
    parents = [draw_parents(k, g, kind) for k in n]
    want = make_tree(parents, n)
    t = api.draft_tree(i32(sum(parents, [])), offsets(n).cuda(), max(n))
    assert torch.equal(t.depths, want.depths) and torch.equal(t.masks, want.masks)
    assert api.read_device_errors() == 0


@gpu
def test_masks_defaults():
    t = api.draft_tree(i32([-1, -1, -1]))                     # one token for each sequence
    assert t.depths.tolist() == [0, 0, 0] and t.masks.tolist() == [[1], [1], [1]]
    t = api.draft_tree(i32([-1, 0, 0, 2]), i32([0, 4]))
    assert t.depths.tolist() == [0, 1, 1, 2] and t.masks.tolist() == [[1], [3], [5], [13]]
    t = api.draft_tree(i32([]), i32([0]))
    assert t.depths.numel() == 0 and t.masks.numel() == 0
    assert api.read_device_errors() == 0


@gpu
def test_masks_flag_what_is_no_tree():
    api.read_device_errors()
    t = api.draft_tree(i32([0, 5, -2, 1, -1, 0]), i32([0, 4, 6]), 4)          # itself, one behind it, below -1
    assert api.read_device_errors() == api.DEVERR_DRAFT
    assert t.depths.tolist() == [0, 0, 0, 1, 0, 1] and t.masks[:, 0].tolist() == [1, 2, 4, 10, 1, 3]
    api.draft_tree(i32([-1, 0, 1, 2]), i32([0, 3, 4]), 2)     # a sequence of more than max_tokens; one of one token, from row 2
    assert api.read_device_errors() == api.DEVERR_LENGTH | api.DEVERR_DRAFT
    for cu in ([1, 4], [0, 3], [0, 9, 4], [0, 3, 1, 4], [0, -7, 4]):
        api.draft_tree(i32([-1, 0, 1, 2]), i32(cu), 4)
        assert api.read_device_errors() & api.DEVERR_LENGTH, cu


# ------------------------------------------------------------------------------------------------ append
@gpu
@pytest.mark.parametrize("H,D,page,block,dt,rot,inter,norm", [
    (2, 128, 64, 16, torch.float32, 128, False, True),
    (1, 64, 16, 16, torch.bfloat16, 64, True, False),
    (3, 64, 96, 32, torch.float16, 32, False, True),
    (2, 256, 64, 64, torch.float32, 256, False, True),
    (1, 256, 32, 16, torch.float16, 0, False, False),
])
@pytest.mark.parametrize("past,n", [([30, 0, 95, 7], [26, 1, 40, 0]), ([0], [1]), ([63, 64, 65], [5, 70, 130])])
def test_append(H, D, page, block, dt, rot, inter, norm, past, n):
    g = torch.Generator().manual_seed(H * D + block + sum(n))
    G = 2 * H
    lens = [a + b for a, b in zip(past, n)]
    cache, table = make_cache(g, lens, H, D, page, block)
    ref = ExactCache(cache)
    parents = [draw_parents(k, g) for k in n]
    tree = make_tree(parents, n)
    rows = (torch.randn(sum(n), G + 2 * H, D, generator=g) * 2).to(dt)
    cos, sin = rotary_tables(max(lens) + 1, rot) if rot else (None, None)
    w = 1 + 0.3 * torch.randn(D, generator=g) if norm else None
    dev = rows.cuda()
    at = offsets(n)
    q = api.kv_append(cache, dev[:, G:G + H], dev[:, G + H:], table.cuda(), i32(lens), at.cuda(),
                      cos.cuda() if rot else None, sin.cuda() if rot else None, inter, w.cuda() if norm else None, 1e-6,
                      dev[:, :G], w.cuda() if norm else None, q_dtype=torch.float32, tree=tree)
    depth = tree.depths.cpu()
    for i, b in enumerate(past):
        lo, hi = int(at[i]), int(at[i + 1])
        if lo == hi:
            continue
        turn = [(cos[b + depth[t]], sin[b + depth[t]]) if rot else (None, None) for t in range(lo, hi)]
        ref.append(0, table[i], b, torch.stack([ref_norm_rope(rows[t, G:G + H], w, 1e-6, *turn[t - lo], inter)
                                                for t in range(lo, hi)]))
        ref.append(1, table[i], b, rows[lo:hi, G + H:])
        for t in range(lo, hi):
            want = ref_norm_rope(rows[t, :G], w, 1e-6, *turn[t - lo], inter)
            assert_close(q[t], want, 16 * 2.0 ** -24 * want.abs().amax(-1, keepdim=True) + 2.0 ** -24 * want.abs() + 1e-7)
    assert_cache(cache, ref, table, lens)
    assert api.read_device_errors() == 0


@gpu
def test_append_of_a_path_is_the_plain_append():
    g = torch.Generator().manual_seed(2)
    n, past = [7, 40, 1], [12, 0, 100]
    lens = [a + b for a, b in zip(past, n)]
    cache, table = make_cache(g, lens, 2, 128, 64, 16)
    other = api.KVCache(*(x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    cos, sin = (t.cuda() for t in rotary_tables(200, 128))
    rows = torch.randn(sum(n), 8, 128, generator=g).cuda()
    tree = make_tree([draw_parents(k, g, "path") for k in n], n)
    args = (rows[:, 4:6], rows[:, 6:], table.cuda(), i32(lens), offsets(n).cuda(), cos, sin)
    a = api.kv_append(cache, *args, q=rows[:, :4])
    b = api.kv_append(other, *args, q=rows[:, :4], tree=tree)
    assert torch.equal(a, b) and all(torch.equal(getattr(cache, x), getattr(other, x)) for x in ("k", "v", "k_scale", "v_scale"))


@gpu
def test_append_flags_depths_outside_the_table():
    g = torch.Generator().manual_seed(3)
    cache, table = make_cache(g, [20], 1, 64, 16, 16)
    x = torch.randn(4, 3, 64, generator=g).cuda()
    cos, sin = (t.cuda() for t in rotary_tables(18, 64))
    tree = make_tree([[-1, 0, 1, 0]], [4])                    # positions 16, 17, 18, 17
    q = torch.full((4, 1, 64), 9.0, device="cuda")
    before = cache.k.clone()
    api.read_device_errors()
    api.kv_append(cache, x[:, 1:2], x[:, 2:], table.cuda(), i32([20]), i32([0, 4]), cos, sin, q=x[:, :1], q_out=q, tree=tree)
    assert api.read_device_errors() == api.DEVERR_POSITION
    assert (q[2] == 9).all() and (q[[0, 1, 3]] != 9).any(-1).all()
    pg = int(table[0, 1])
    assert torch.equal(cache.k[pg, 0, 2], before[pg, 0, 2]) and not torch.equal(cache.k[pg, 0, 3], before[pg, 0, 3])


# ------------------------------------------------------------------------------------------------ attention
def ref_tree_attention(q, cache, table, lens, n, masks, scale, window):
    """masks: for each sequence, bool [n, n]."""
    ref = RefCache(cache)
    T, Hq, D = q.shape
    group = Hq // cache.kv_heads
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    vmax, at = 0.0, 0
    for i, (L, m) in enumerate(zip(lens, n)):
        if m and L:
            k, v = (ref.values(side, table[i], 0, L) for side in (0, 1))
            vmax = max(vmax, float(v.abs().max()))
            first = L - m
            see = torch.ones(m, L, dtype=torch.bool)
            see[:, max(first, 0):] = masks[i][:, max(-first, 0):]
            if window:
                place = first + masks[i].sum(-1, keepdim=True) - 1
                see &= (torch.arange(L)[None] > place - window) | (torch.arange(L)[None] >= first)
            for h in range(Hq):
                s = (q[at:at + m, h].double() @ k[:, h // group].T * scale).masked_fill(~see, -math.inf)
                top = s.amax(-1, keepdim=True)
                p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
                z = p.sum(-1, keepdim=True)
                out[at:at + m, h] = (p / torch.where(z > 0, z, torch.ones_like(z))) @ v[:, h // group]
                lse[at:at + m, h] = (torch.log(z) + top)[:, 0]
        at += m
    return out, lse, vmax


@pytest.fixture(params=["close", "loose"])
def bound(request, monkeypatch):
    """Which kernel takes the rows depends on the bounds of the lengths: with a loose one, short sequences take the one that
    long ones take."""
    monkeypatch.setattr(sys.modules[__name__], "BOUND", 1 << 20 if request.param == "loose" else None)


BOUND = None


def top(lens):
    return BOUND or max(lens)


def check(past, n, Hq, H, D, page=64, block=16, qt=torch.bfloat16, ot=torch.float32, window=0, scale=None, kind="any",
          spread=1.0, tamper=None, seed=0, no_cu=False, **more):
    lens = [max(a + b, 0) for a, b in zip(past, n)]
    g = torch.Generator().manual_seed(seed + sum(lens) + D)
    cache, table = make_cache(g, lens, H, D, page, block)
    q = (torch.randn(sum(n), Hq, D, generator=g) * spread).to(qt)
    if tamper:
        tamper(cache, table, q)
    parents = [draw_parents(k, g, kind) for k in n]
    scale = D ** -0.5 if scale is None else scale
    want, wlse, vmax = ref_tree_attention(q, cache, table, lens, n, [sees(p) for p in parents], scale, window)
    api.read_device_errors()
    out, lse = api.attention(q.cuda(), cache, table.cuda(), i32(lens), max_kv_len=top(lens),
                             cu_tokens=None if no_cu else offsets(n).cuda(), max_tokens=max(n), scale=scale,
                             window=window, out_dtype=ot, return_lse=True, tree=make_tree(parents, n), **more)
    tol = vmax * (2.0 ** -11 + 2.0 ** -16 + ULP[ot])
    assert_close(out, want, torch.full_like(want, tol), "out")
    empty = wlse == -math.inf
    assert torch.equal(torch.isneginf(lse).cpu(), empty)
    assert (out.cpu()[empty] == 0).all()
    err = (lse.double().cpu() - wlse)[~empty].abs()
    assert (err <= 2.0 ** -18 + 2.0 ** -20 * wlse[~empty].abs()).all(), float(err.max())
    assert api.read_device_errors() == 0


SHAPES = [(4, 4, 64, 16, 16), (8, 2, 128, 64, 16), (7, 1, 128, 32, 32), (16, 1, 64, 64, 64), (6, 2, 256, 48, 16),
          (10, 2, 256, 64, 64), (3, 1, 128, 128, 32)]


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("Hq,H,D,page,block", SHAPES)
@pytest.mark.parametrize("past,n", [([0], [1]), ([0], [5]), ([1, 15, 16, 17], [1, 2, 3, 4]), ([127, 128, 129], [1, 9, 30]),
                                    ([100, 255, 0, 250], [28, 1, 64, 26]), ([700, 64, 0], [40, 129, 70]),
                                    ([300, 5], [0, 200])])
def test_attention(Hq, H, D, page, block, past, n):
    check(past, n, Hq, H, D, page, block, torch.float16 if D == 64 else torch.bfloat16)


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("kind", ["forest", "path", "star", "apart"])
def test_attention_kinds_of_trees(kind):
    check([130, 0, 61], [33, 12, 97], 8, 2, 128, kind=kind)
    check([130, 0, 61], [33, 12, 97], 6, 2, 64, 32, 32, kind=kind)


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("past,n", [([5000, 150, 2311], [9, 20, 33]), ([9001], [26]), ([20011, 1025, 30], [3, 60, 140]),
                                    ([40000], [2])])
def test_attention_split_along_the_cache(D, past, n):
    check(past, n, 4, 1, D, 64, 16)


@gpu
@pytest.mark.usefixtures("bound")
def test_attention_of_many_sequences():
    g = torch.Generator().manual_seed(5)
    n = torch.randint(0, 6, (1300,), generator=g).tolist()
    past = torch.randint(0, 40, (1300,), generator=g).tolist()
    check(past, n, 4, 2, 64, 16, 16)
    check(past, n, 16, 2, 64, 16, 16)
    check([3] * 600, [1] * 600, 2, 1, 128, 16, 16, no_cu=True)
    check([3] * 600, [1] * 600, 20, 1, 128, 16, 16, no_cu=True)


@gpu
def test_attention_of_more_tiles_than_a_block_lists_at_once(monkeypatch):
    """Units that lie across two lists of a block among them."""
    monkeypatch.setattr(sys.modules[__name__], "BOUND", 1 << 20)
    g = torch.Generator().manual_seed(9)
    n = torch.randint(0, 4, (3300,), generator=g).tolist()
    past = torch.randint(0, 500, (3300,), generator=g).tolist()
    check(past, n, 16, 2, 64, 16, 16)


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_of_one_large_tree_among_small_ones(D):
    check([50] + [20] * 40, [300] + [1, 2] * 20, 8, 1, D, 16, 16)


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("n", [3, 12, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_rows_that_are_no_numbers_stay_alone(n, D):
    """A row of NaN, of an infinity, of zeros, of the largest values: the other rows are what they are without them."""
    g = torch.Generator().manual_seed(3)
    cache, table = make_cache(g, [300], 2, D, 64, 16)
    q = torch.randn(n, 8, D, generator=g).bfloat16()
    tree = make_tree([draw_parents(n, g)], [n])
    args = (cache, table.cuda(), i32([300]), top([300]), i32([0, n]), n)
    vmax = float((cache.v.abs().amax((2, 3)) * cache.v_scale.amax(-1)).max())
    for small in (1.0, 2.0 ** -20):                           # small rows under a large scale: only the whole has to be in bounds
        more = dict(scale=D ** -0.5 / small, out_dtype=torch.float32, tree=tree)
        want = api.attention((q * small).cuda(), *args, **more)
        for value in (float("nan"), float("inf"), -float("inf"), 0.0) + ((3.0e38,) if small == 1.0 else ()):
            x = q * small
            x[1, 3, 5] = value
            x[2, 6] = value
            got = api.attention(x.cuda(), *args, **more)
            same = torch.ones(n, 8, dtype=torch.bool)
            same[1, 3] = same[2, 6] = False
            assert (got - want).abs()[same.cuda()].max() <= 2 * vmax * (2.0 ** -11 + 2.0 ** -16), (value, small)
            if value == 0.0:
                assert torch.isfinite(got).all()
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.usefixtures("bound")
def test_attention_two_calls_at_once():
    g = torch.Generator().manual_seed(6)
    calls = []
    for lens, n, D in (([3000, 200, 900], 20, 128), ([5000, 77], 11, 64)):
        cache, table = make_cache(g, lens, 2, D, 64, 16)
        q = torch.randn(n * len(lens), 8, D, generator=g).bfloat16().cuda()
        tree = make_tree([draw_parents(n, g) for _ in lens], [n] * len(lens))
        calls.append((q, cache, table.cuda(), i32(lens), top(lens), offsets([n] * len(lens)).cuda(), n, tree))
    want = [api.attention(*c[:-1], tree=c[-1]) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for c, st, o in zip(calls, streams, got):
            with torch.cuda.stream(st):
                o.append(api.attention(*c[:-1], tree=c[-1]))
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(w, x) for x in o)


@gpu
@pytest.mark.usefixtures("bound")
def test_attention_of_the_largest_trees():
    check([100, 0], [1024, 1000], 2, 1, 64, 64, 16)
    check([1000], [1024], 3, 1, 128, 64, 64, kind="path")


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("window", [64, 70, 100, 300, 5000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_window(window, D):
    check([400, 150, 33, 2000], [64, 3, 30, 10], 8, 2, D, 32, 16, window=window)


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_rows_without_a_place(D):
    """Sequences shorter than their new tokens: the first tokens have no place, rows that see only these see nothing."""
    check([-3, 5, -40], [4, 7, 100], 8, 2, D, 32, 16)
    check([-3, -1], [4, 1], 8, 2, D, 32, 16, kind="apart")


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("qt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ot", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [[2, 3], [70, 20]])
def test_attention_types(qt, ot, n):
    check([200, 77], n, 8, 4, 128, 64, 32, qt, ot)


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("n", [[2, 1], [3, 100]])
def test_attention_sharp_rows_and_scales(n):
    """Scores far apart, queries of extreme bf16 magnitude, zero value blocks, scales of many magnitudes."""
    def tamper(cache, table, q):
        q[0] *= 8.0
        cache.v_scale[int(table[0, 0]), :, 0] = 0
        cache.v[int(table[0, 0]), :, :16] = 0
        cache.v_scale[int(table[0, 2])] = 1e-7
        cache.k_scale[int(table[1, 0]), :, 0] = 0
    check([300, 200], n, 8, 2, 128, 64, 16, tamper=tamper)

    def tiny(cache, table, q):
        q *= 2.0 ** -100
        cache.v_scale.mul_(2.0 ** -30)
    check([300, 200], n, 8, 2, 64, 64, 16, tamper=tiny, scale=2.0 ** 97)
    check([300, 200], n, 8, 2, 64, 64, 16, scale=-0.1)
    check([300, 200], n, 8, 2, 256, 64, 16, scale=0.0)


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_reference_that_grows_late(D):
    """Keys whose scores rise along the cache, so that the running reference is raised again and again."""
    def tamper(cache, table, q):
        q.abs_()
        cache.k.copy_(torch.randint(60, 70, cache.k.shape, generator=torch.Generator().manual_seed(1)))
        for j, pg in enumerate(table[0].tolist()):
            if pg >= 0:
                cache.k_scale[pg] = 0.002 * (j + 1)
    check([1000], [20], 8, 2, D, 64, 16, tamper=tamper)
    check([1000], [20], 8, 2, D, 64, 16, tamper=tamper, scale=-D ** -0.5)


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("n", [[2, 3], [30, 100]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_ignores_what_lies_past_the_length(n, D):
    """NaN scales and any codes past the length, invalid table entries and mask bits past the tokens change nothing."""
    g = torch.Generator().manual_seed(5)
    lens = [290, 163]
    cache, table = make_cache(g, lens, 2, D, 64, 16)
    q = torch.randn(sum(n), 8, D, generator=g).bfloat16().cuda()
    tree = make_tree([draw_parents(k, g) for k in n], n)
    args = (i32(lens), top(lens), offsets(n).cuda(), max(n))
    first = api.attention(q, cache, table.cuda(), *args, tree=tree)
    used = torch.zeros(cache.pages, 64, dtype=torch.bool)
    for i, L in enumerate(lens):
        at = torch.arange(L)
        used[table[i][at // 64].long(), at % 64] = True
    dead = (~used).cuda()
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.permute(0, 2, 1, 3)[dead] = -128
        s.permute(0, 2, 1)[dead.view(cache.pages, 4, 16).all(-1)] = float("nan")
    table[:, -1] = 2 ** 30
    wider = torch.full((sum(n), tree.masks.shape[1] + 1), -1, dtype=torch.int32, device="cuda")
    wider[:, :-1] = tree.masks
    for i, k in enumerate(n):
        bits = (1 << 32) - (1 << (k % 32)) if k % 32 else 0
        if bits and k // 32 < tree.masks.shape[1]:
            wider[sum(n[:i]):sum(n[:i]) + k, k // 32] |= bits - (1 << 32)
    again = api.attention(q, cache, table.cuda(), *args, tree=api.DraftTree(tree.depths, wider))
    assert torch.equal(first, again)
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.usefixtures("bound")
@pytest.mark.parametrize("n", [2, 50])
def test_attention_strided_rows_streams_and_workspace(n):
    """Queries and outputs that are slices of wider rows, another stream, a caller's workspace: the same bits."""
    g = torch.Generator().manual_seed(11)
    lens = [3000, 2900]
    cache, table = make_cache(g, lens, 2, 128, 64, 32)
    wide = torch.randn(2 * n, 13, 128, generator=g).bfloat16().cuda()
    q = wide[:, 2:10]
    tree = make_tree([draw_parents(n, g), draw_parents(n, g)], [n, n])
    kv, cu, tb = i32(lens), offsets([n, n]).cuda(), table.cuda()
    want = api.attention(q.contiguous(), cache, tb, kv, top(lens), cu, n, tree=tree)
    need = api.attention_tree_workspace_bytes(2 * n, 8, 2, 128, 2, n, top(lens))
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((2 * n, 12, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    api.attention(q, cache, tb, kv, top(lens), cu, n, out=out[:, 1:9], workspace=ws, stream=st, tree=tree)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out[:, 1:9], want)
    assert (out[:, 0] == 5).all() and (out[:, 9:] == 5).all() and (ws[need:] == 0xFF).all()


@gpu
@pytest.mark.parametrize("n,Hq,H,D", [(2, 4, 1, 64), (60, 4, 1, 64), (100, 32, 8, 256)])
def test_attention_flags_lengths_pages_and_offsets(n, Hq, H, D):
    g = torch.Generator().manual_seed(2)
    cache, table = make_cache(g, [300], H, D, 64, 16)
    q = torch.randn(n, Hq, D, generator=g).bfloat16().cuda()
    tree = make_tree([draw_parents(n, g)], [n])
    cu, kv = i32([0, n]), i32([300])
    api.read_device_errors()
    api.attention(q, cache, table.cuda(), kv, 200, cu, n, tree=tree)
    assert api.read_device_errors() == api.DEVERR_LENGTH
    out = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    api.attention(q, cache, table.cuda(), kv, 300, cu, n - 1, out=out, tree=tree)         # one token more than stated
    assert api.read_device_errors() == api.DEVERR_LENGTH
    assert (out[n - 1:] == 7).all() and (out[:n - 1] != 7).any(-1).all()
    for offset in ([0, n - 1], [1, n], [0, n + 5]):
        api.attention(q, cache, table.cuda(), kv, 300, i32(offset), n, tree=tree)
        assert api.read_device_errors() & api.DEVERR_LENGTH, offset
    table[0, 1] = -5
    out = api.attention(q, cache, table.cuda(), kv, 300, cu, n, tree=tree)
    assert api.read_device_errors() == api.DEVERR_PAGE and torch.isfinite(out.float()).all()


@gpu
@pytest.mark.parametrize("n", [5, 16])
def test_attention_of_a_batch_flags_lengths_pages_and_offsets(n):
    """As above, where the tiles of many sequences are shared out."""
    g = torch.Generator().manual_seed(2)
    S = 128
    cache, table = make_cache(g, [300] * S, 8, 128, 64, 16)
    q = torch.randn(S * n, 32, 128, generator=g).bfloat16().cuda()
    tree = make_tree([draw_parents(n, g) for _ in range(S)], [n] * S)
    tb, kv, cu = table.cuda(), i32([300] * S), offsets([n] * S).cuda()
    api.read_device_errors()
    want = api.attention(q, cache, tb, kv, 300, cu, n, tree=tree)
    assert api.read_device_errors() == 0
    api.attention(q, cache, tb, kv, 250, cu, n, tree=tree)
    assert api.read_device_errors() == api.DEVERR_LENGTH
    out = torch.full((S, n, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    api.attention(q, cache, tb, kv, 300, cu, n - 1, out=out.view(S * n, 32, 128), tree=tree)     # one token more than stated
    assert api.read_device_errors() == api.DEVERR_LENGTH
    assert (out[:, n - 1] == 7).all() and (out[:, :n - 1] != 7).any(-1).all()
    for last in (S * n - 1, S * n + 5):
        wrong = cu.clone()
        wrong[-1] = last
        api.attention(q, cache, tb, kv, 300, wrong, n + 5, tree=tree)
        assert api.read_device_errors() & api.DEVERR_LENGTH, last
    fallen = cu.clone()
    fallen[40] = 0
    api.attention(q, cache, tb, kv, 300, fallen, n, tree=tree)
    assert api.read_device_errors() & api.DEVERR_LENGTH
    table[3, 1], table[77, 4] = -5, 2 ** 30
    got = api.attention(q, cache, table.cuda(), kv, 300, cu, n, tree=tree)
    assert api.read_device_errors() == api.DEVERR_PAGE and torch.isfinite(got.float()).all()
    others = torch.ones(S, dtype=torch.bool)
    others[3] = others[77] = False
    vmax = float((cache.v.abs().amax((2, 3)) * cache.v_scale.amax(-1)).max())
    diff = (got.float() - want.float()).view(S, -1).abs().amax(-1).cpu()
    assert diff[others].max() <= vmax * (2 * (2.0 ** -11 + 2.0 ** -16) + 2.0 ** -7) and (diff[~others] > 0).all()


@gpu
@pytest.mark.usefixtures("bound")
def test_attention_of_a_path_is_causal_attention():
    g = torch.Generator().manual_seed(8)
    n, lens = [5, 33, 1], [800, 33, 400]
    cache, table = make_cache(g, lens, 2, 128, 64, 16)
    q = torch.randn(sum(n), 8, 128, generator=g).bfloat16().cuda()
    args = (q, cache, table.cuda(), i32(lens), top(lens), offsets(n).cuda(), max(n))
    a, la = api.attention(*args, out_dtype=torch.float32, return_lse=True)
    b, lb = api.attention(*args, out_dtype=torch.float32, return_lse=True,
                          tree=make_tree([draw_parents(k, g, "path") for k in n], n))
    vmax = float((cache.v.abs().amax((2, 3)) * cache.v_scale.amax(-1)).max())
    assert (a - b).abs().max() <= vmax * 2 * (2.0 ** -11 + 2.0 ** -16) and (la - lb).abs().max() <= 2.0 ** -17 + 2.0 ** -19 * 12


# ------------------------------------------------------------------------------------------------ keep
def ref_keep(cache, table, lens, n, kept):
    """Codes and scales after the call, to the bit; f32 arithmetic as it is defined."""
    codes, scale = [cache.k.cpu(), cache.v.cpu()], [cache.k_scale.cpu(), cache.v_scale.cpu()]
    B, P = cache.block, cache.page_size
    for i, rows in enumerate(kept):
        base = lens[i] - n[i]
        still = sum(1 for j, r in enumerate(rows) if r == j)
        if still == len(rows):
            continue
        for c, s in zip(codes, scale):
            old_c, old_s = c.clone(), s.clone()
            for b in range((base + still) // B, (base + len(rows) - 1) // B + 1):
                to = range(b * B, min(b * B + B, base + len(rows)))
                src = [p if p < base else base + rows[p - base] for p in to]
                was = torch.stack([old_s[int(table[i, p // P]), :, p % P // B] for p in src])
                top = was.amax(0)
                ratio = torch.where(top > 0, was / torch.where(top > 0, top, torch.ones_like(top)), torch.zeros_like(was))
                for k, (p, f) in enumerate(zip(to, src)):
                    x = old_c[int(table[i, f // P]), :, f % P].float()
                    c[int(table[i, p // P]), :, p % P] = torch.round(x * ratio[k][:, None]).to(torch.int8)
                s[int(table[i, b * B // P]), :, b * B % P // B] = top
    return codes, scale


def check_keep(past, n, kept, H, D, page, block, seed=0, zero=False):
    lens = [a + b for a, b in zip(past, n)]
    g = torch.Generator().manual_seed(seed + sum(lens) + D)
    cache, table = make_cache(g, lens, H, D, page, block)
    if zero:
        cache.k_scale.zero_()
        cache.k.zero_()
    codes, scale = ref_keep(cache, table, lens, n, kept)
    most = max(len(r) for r in kept) + 1
    rows = i32([r + [-9] * (most - len(r)) for r in kept])
    api.read_device_errors()
    api.kv_keep(cache, table.cuda(), i32(lens), sum(n), rows, i32([len(r) for r in kept]), offsets(n).cuda())
    for i, (b, r) in enumerate(zip(past, kept)):              # past the kept tokens: undefined
        at = torch.arange(b + len(r))
        pg, off = table[i][at // page].long(), at % page
        for got, want, gs, ws in zip((cache.k, cache.v), codes, (cache.k_scale, cache.v_scale), scale):
            assert torch.equal(got.cpu()[pg, :, off], want[pg, :, off]), i
            assert torch.equal(gs.cpu()[pg, :, off // block], ws[pg, :, off // block]), i
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("H,D,page,block", [(2, 128, 64, 16), (1, 64, 16, 16), (3, 64, 96, 32), (2, 256, 64, 64),
                                            (1, 256, 32, 16), (8, 128, 64, 64), (2, 256, 128, 32)])
def test_keep(H, D, page, block):
    g = torch.Generator().manual_seed(H * D)
    past, n = [0, 31, 700, 16, 5, 63, 48], [26, 40, 130, 1, 9, 70, 300]
    kept = [[0, 3, 7, 20], [0, 1, 2], [0, 2] + list(range(40, 130, 3)), [0], [], [69], list(range(0, 300, 2))]
    check_keep(past, n, kept, H, D, page, block)
    kept = [sorted(torch.randperm(k, generator=g)[:max(1, k // 3)].tolist()) for k in n]
    check_keep(past, n, kept, H, D, page, block, 1)
    check_keep(past, n, [list(range(k)) for k in n], H, D, page, block, 2)
    check_keep(past, n, kept, H, D, page, block, 3, zero=True)


@gpu
def test_keep_of_a_long_path():
    check_keep([77, 1000], [1024, 1023], [list(range(0, 1024, 1))[1:], list(range(200, 1023))], 1, 64, 64, 16)


@gpu
def test_keep_refuses_rows_that_are_no_path():
    g = torch.Generator().manual_seed(9)
    n, lens = [6] * 6, [30] * 6
    cache, table = make_cache(g, lens, 2, 64, 16, 16)
    before = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    rows = i32([[0, 2, 2], [3, 1, 5], [0, 4, 6], [-1, 2, 3], [0, 2, 4], [0, 1, 2]])
    api.read_device_errors()
    for counts in ([3, 3, 3, 3, 4, -1], [3, 2, 3, 1, 7, 1 << 30]):
        api.kv_keep(cache, table.cuda(), i32(lens), 36, rows, i32(counts), offsets(n).cuda())
        assert api.read_device_errors() == api.DEVERR_DRAFT
    api.kv_keep(cache, table.cuda(), i32([3] * 6), 36, rows, i32([3] * 6), offsets(n).cuda())     # shorter than its tokens
    assert api.read_device_errors() == api.DEVERR_LENGTH
    api.kv_keep(cache, table[:, :1].contiguous().cuda(), i32(lens), 36, rows, i32([3] * 6), offsets(n).cuda())
    assert api.read_device_errors() == api.DEVERR_LENGTH
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    api.kv_keep(cache, table.cuda(), i32(lens), 6, i32([[0]] * 6), i32([1] * 6))                  # one token each: stays
    assert api.read_device_errors() == 0
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


@gpu
def test_keep_with_invalid_pages():
    g = torch.Generator().manual_seed(9)
    cache, table = make_cache(g, [40], 1, 64, 16, 16)
    held = [x.clone() for x in (cache.k, cache.k_scale)]
    bad = table.clone()
    bad[0, 2] = cache.pages                                   # tokens 32.. have no place: they become zeros
    api.read_device_errors()
    api.kv_keep(cache, bad.cuda(), i32([40]), 30, i32([[0, 5, 25]]), i32([3]), i32([0, 30]))
    assert api.read_device_errors() == api.DEVERR_PAGE
    pg = int(table[0, 0])
    assert torch.equal(cache.k[pg, 0, 11], held[0][pg, 0, 15]) and (cache.k[pg, 0, 12] == 0).all()
    assert torch.equal(cache.k[pg, 0, :11], held[0][pg, 0, :11]) and torch.equal(cache.k_scale, held[1])


# ------------------------------------------------------------------------------------------------ together
@gpu
@pytest.mark.parametrize("D,page,block", [(64, 32, 32), (128, 64, 16), (256, 64, 64)])
def test_verification_steps(D, page, block):
    """Several steps over one cache, as a server runs them: each drafts a tree, scores it and keeps a path; the accepted
    tokens' keys and values must be those that appends of the paths alone would have left, to the steps of the codes."""
    g = torch.Generator().manual_seed(D)
    H, Hq, S = 2, 6, 3
    cos, sin = (t.cuda() for t in rotary_tables(400, D))
    wk = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    cache, table = make_cache(g, [300] * S, H, D, page, block, fill=False)
    tb = table.cuda()
    lens = [40, 3, 0]
    text = [torch.randn(L, Hq + 2 * H, D, generator=g).cuda() for L in lens]
    rows = torch.cat(text)
    api.kv_append(cache, rows[:, Hq:Hq + H], rows[:, Hq + H:], tb, i32(lens), offsets(lens).cuda(), cos, sin, k_weight=wk)
    for step in range(4):
        n = [26, 1 + 11 * step, 33]
        parents = [draw_parents(k, g) for k in n]
        rows = (torch.randn(sum(n), Hq + 2 * H, D, generator=g) * 1.2).cuda()
        grown = [a + b for a, b in zip(lens, n)]
        cu = offsets(n).cuda()
        tree = api.draft_tree(i32(sum(parents, [])), cu, max(n))
        q = api.kv_append(cache, rows[:, Hq:Hq + H], rows[:, Hq + H:], tb, i32(grown), cu, cos, sin, k_weight=wk,
                          q=rows[:, :Hq], q_dtype=torch.bfloat16, tree=tree)
        out = api.attention(q, cache, tb, i32(grown), max(grown), cu, max(n), out_dtype=torch.float32, tree=tree)
        masks = [sees(p) for p in parents]
        want, _, vmax = ref_tree_attention(q.cpu(), cache, table, grown, n, masks, D ** -0.5, 0)
        assert_close(out, want, torch.full_like(want, vmax * (2.0 ** -11 + 2.0 ** -16)), f"step {step}")
        kept = []
        for i, m in enumerate(masks):
            leaf = int(torch.randint(0, n[i], (1,), generator=g))
            kept.append(m[leaf].nonzero().flatten().tolist())
            at = int(cu[i])
            text[i] = torch.cat([text[i], rows[at:at + n[i]][kept[-1]]])
        most = max(map(len, kept))
        api.kv_keep(cache, tb, i32(grown), sum(n), i32([r + [0] * (most - len(r)) for r in kept]),
                    i32([len(r) for r in kept]), cu)
        lens = [a + len(r) for a, r in zip(lens, kept)]
    k, v = api.kv_read(cache, tb, i32(lens), sum(lens), offsets(lens).cuda(), torch.float32)
    at = offsets(lens)
    for i, L in enumerate(lens):
        x = text[i]
        pos = torch.arange(L, dtype=torch.int32, device="cuda")
        _, rk = api.qk_norm_rope(None, x[:, Hq:Hq + H], pos, cos, sin, k_weight=wk)
        for got, ref in ((k, rk), (v, x[:, Hq + H:])):
            # two roundings a step of at most half a code each, the scale at most that of the largest value drafted
            err = (got[at[i]:at[i + 1]] - ref).abs().max()
            assert err <= 8 * 1.2 * 5.5 / 127, float(err)
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.usefixtures("bound")
def test_steps_in_a_graph():
    """A captured step replays while lengths, trees and paths change on the device."""
    g = torch.Generator().manual_seed(4)
    H, Hq, D, S, n = 2, 8, 128, 3, 20
    cache, table = make_cache(g, [700] * S, H, D, 64, 16, fill=False)
    tb, cu = table.cuda(), offsets([n] * S).cuda()
    cos, sin = (t.cuda() for t in rotary_tables(800, D))
    rows = torch.zeros(S * n, Hq + 2 * H, D, device="cuda")
    parents, kept, counts = i32([-1] * (S * n)), i32([[0] * 6] * S), i32([1] * S)
    lens = i32([0] * S)
    q = torch.empty(S * n, Hq, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(S * n, Hq, D, device="cuda")
    ws = torch.empty(api.attention_tree_workspace_bytes(S * n, Hq, H, D, S, n, top([700])) + 16, dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(n)
        tree = api.draft_tree(parents, cu, n)
        api.kv_append(cache, rows[:, Hq:Hq + H], rows[:, Hq + H:], tb, lens, cu, cos, sin, q=rows[:, :Hq], q_out=q, tree=tree)
        api.attention(q, cache, tb, lens, top([700]), cu, n, out=out, workspace=ws, tree=tree)

    def accept():
        api.kv_keep(cache, tb, lens, S * n, kept, counts, cu)
        lens.add_(counts - n)

    step()
    accept()
    graphs = []
    for f in (step, accept):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    lens.zero_()
    total = [0] * S
    for i in range(25):
        p = [draw_parents(n, g, "forest" if i % 2 else "any") for _ in range(S)]
        rows.copy_(torch.randn(rows.shape, generator=g))
        parents.copy_(i32(sum(p, [])))
        graphs[0].replay()
        if i % 8 == 7:
            grown = [t + n for t in total]
            assert lens.tolist() == grown
            want, _, vmax = ref_tree_attention(q.cpu(), cache, table, grown, [n] * S, [sees(x) for x in p], D ** -0.5, 0)
            assert_close(out, want, torch.full_like(want, vmax * (2.0 ** -11 + 2.0 ** -16)))
        path = [sees(x)[-1].nonzero().flatten().tolist()[:6] for x in p]
        kept.copy_(i32([r + [0] * (6 - len(r)) for r in path]))
        counts.copy_(i32([len(r) for r in path]))
        graphs[1].replay()
        total = [t + len(r) for t, r in zip(total, path)]
        assert lens.tolist() == total
    assert api.read_device_errors() == 0
