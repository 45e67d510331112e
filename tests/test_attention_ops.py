"""Attention over the 8-bit paged cache and the operators around it, against plain 64-bit implementations.

Tolerances, from the arithmetic:
  norm_rope   f32 throughout: a sum of D <= 256 squares, rsqrt (2 ulp), three products and a rotation: below
              16 * 2^-24 of the head's largest output magnitude, plus half an ulp of the output type.
  append      the code is round(x / s): the kernel's f32 x differs from the 64-bit one by some 2^-21 of the block's
              largest magnitude, so a code may differ by one step where x / s is that close to a half; the scale agrees
              to 2^-21.  Values are compared to one step, and at most 1 in 1000 may differ by more than 2^-18 of it.
  attention   probabilities as fp16 (2^-11 each) over values of magnitude <= vmax: 2^-11 vmax plus half an ulp of
              the output type; queries and scores carry 2^-22 relative, scores here stay below 2^5: 2^-16 of vmax.
              lse: f32, 2^-18 absolute + 2^-20 relative.
"""
import math

import numpy as np
import pytest
import torch

from block_quantized_int8_q8_gb300 import api

gpu = pytest.mark.gpu
ULP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}      # half an ulp at 1


def rotary_tables(n, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * inv
    return torch.from_numpy(np.cos(a)).float(), torch.from_numpy(np.sin(a)).float()


def ref_norm_rope(x, w, eps, cos, sin, interleaved):
    """x [H, D], one token, in 64 bits; cos, sin [rot/2] or None."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if cos is None:
        return x
    y = x.clone()
    half = cos.numel()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[:, a] = x[:, a] * cos[i].double() - x[:, b] * sin[i].double()
        y[:, b] = x[:, a] * sin[i].double() + x[:, b] * cos[i].double()
    return y


def assert_close(got, ref, tol, what=""):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got.double()).all(), what
    assert (err <= tol).all(), f"{what}: {float((err - tol).max())} over its tolerance (error {float(err.max())})"


# ------------------------------------------------------------------------------------------------ norm_rope
@gpu
@pytest.mark.parametrize("dim,hq,hk,rot,inter,it,ot,norm", [
    (128, 32, 8, 128, False, torch.float32, torch.bfloat16, True),
    (128, 5, 1, 64, True, torch.bfloat16, torch.bfloat16, True),
    (64, 3, 3, 64, True, torch.float16, torch.float32, False),
    (64, 12, 4, 8, False, torch.bfloat16, torch.float16, True),
    (256, 7, 1, 256, False, torch.float32, torch.float32, True),
    (256, 2, 2, 64, False, torch.float16, torch.float16, False),
])
@pytest.mark.parametrize("tokens", [1, 3, 67])
def test_norm_rope(dim, hq, hk, rot, inter, it, ot, norm, tokens):
    g = torch.Generator().manual_seed(dim + tokens)
    rows = (torch.randn(tokens, hq + 2 * hk, dim, generator=g) * 2).to(it)
    rows[0, 0] = 0                                            # a zero head stays zero
    wq, wk = (1 + 0.3 * torch.randn(dim, generator=g) for _ in range(2))
    cos, sin = rotary_tables(500, rot)
    pos = torch.randint(0, 500, (tokens,), generator=g, dtype=torch.int32)
    dev = rows.cuda()
    q, k = dev[:, :hq], dev[:, hq:hq + hk]
    before = dev.clone()
    qo, ko = api.qk_norm_rope(q, k, pos.cuda(), cos.cuda(), sin.cuda(), wq.cuda() if norm else None,
                              wk.cuda() if norm else None, 1e-6, inter, dtype=ot)
    assert qo.dtype == ot and torch.equal(dev, before)
    for x, o, w in ((rows[:, :hq], qo, wq), (rows[:, hq:hq + hk], ko, wk)):
        for t in range(tokens):
            ref = ref_norm_rope(x[t], w if norm else None, 1e-6, cos[pos[t]], sin[pos[t]], inter)
            tol = 16 * 2.0 ** -24 * ref.abs().amax(-1, keepdim=True) + ULP[ot] * ref.abs() + 1e-7
            assert_close(o[t], ref, tol, f"token {t}")
    if it == ot:                                              # in place, within the fused rows; the rest untouched
        api.qk_norm_rope(q, k, pos.cuda(), cos.cuda(), sin.cuda(), wq.cuda() if norm else None,
                         wk.cuda() if norm else None, 1e-6, inter, q_out=q, k_out=k)
        assert torch.equal(q, qo) and torch.equal(k, ko)
        assert torch.equal(dev[:, hq + hk:], before[:, hq + hk:])
    assert api.read_device_errors() == 0


@gpu
def test_norm_rope_one_side_and_norm_only():
    x = torch.randn(9, 6, 128, device="cuda")
    w = torch.rand(128, device="cuda") + 0.5
    q, k = api.qk_norm_rope(x, None, q_weight=w)
    q2, k2 = api.qk_norm_rope(None, x, k_weight=w)
    assert k is None and q2 is None and torch.equal(q, k2)
    ref = torch.stack([ref_norm_rope(x[t].cpu(), w.cpu(), 1e-6, None, None, False) for t in range(9)])
    assert_close(q, ref, 16 * 2.0 ** -24 * ref.abs().amax() + 1e-7)


@gpu
def test_norm_rope_position_outside_the_table_is_flagged_and_skipped():
    x = torch.randn(3, 2, 64, device="cuda")
    cos, sin = (t.cuda() for t in rotary_tables(10, 64))
    out = torch.full_like(x, 7.0)
    api.read_device_errors()
    api.qk_norm_rope(x, None, torch.tensor([3, 10, -1], dtype=torch.int32, device="cuda"), cos, sin, q_out=out)
    assert api.read_device_errors() == api.DEVERR_POSITION
    assert (out[1:] == 7).all() and (out[0] != 7).any()


# ------------------------------------------------------------------------------------------------ the cache
class RefCache:
    """Blocks of values in 64 bits, from the definition: {(page, head, block): (scale, codes [block, D])} lazily."""

    def __init__(self, cache):
        self.c = cache
        self.codes = [cache.k.cpu().double(), cache.v.cpu().double()]
        self.scale = [cache.k_scale.cpu().double(), cache.v_scale.cpu().double()]

    def append(self, side, row, start, x):
        """x [n, H, D] at positions start.. of the sequence with page table row `row`."""
        c, s, B, P = self.codes[side], self.scale[side], self.c.block, self.c.page_size
        n = x.shape[0]
        for b in range(max(start, 0) // B, -(-(start + n) // B)):
            pg, off = int(row[b * B // P]), b * B % P
            lo, hi = max(start, b * B), min(start + n, b * B + B)
            new = x[lo - start:hi - start].double()
            need = (new.abs().amax((0, 2)) / 127).float().double()        # the cache holds f32 scales
            need = torch.where(need < 2.0 ** -63, torch.zeros_like(need), need)
            old = torch.zeros_like(need) if lo == b * B else s[pg, :, off // B]
            d = torch.maximum(old, need)
            safe = torch.where(d > 0, d, torch.ones_like(d))[:, None, None]
            held = c[pg, :, off:off + lo - b * B]
            c[pg, :, off:off + lo - b * B] = torch.round(held * old[:, None, None] / safe)
            c[pg, :, off + lo - b * B:off + hi - b * B] = torch.round(new.transpose(0, 1) / safe).clamp(-127, 127)
            s[pg, :, off // B] = d

    def values(self, side, row, lo, hi):
        c, s, B, P = self.codes[side], self.scale[side], self.c.block, self.c.page_size
        at = torch.arange(lo, hi)
        pg = torch.as_tensor(row)[at // P].long()
        return c[pg, :, at % P] * s[pg, :, at % P // B][..., None]


def make_cache(g, lens, H, D, page, block, fill=True):
    per = [-(-n // page) for n in lens]
    total = sum(per) + 2
    cache = api.KVCache.empty(total, H, D, page, block)
    if fill:
        for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            c.copy_((torch.randn(c.shape, generator=g) * 40).round().clamp(-127, 127))
            s.copy_(torch.rand(s.shape, generator=g) * 0.04 + 0.001)
    else:                                                     # unwritten memory may hold anything
        for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            c.fill_(-128)
            s.fill_(float("nan"))
    order = torch.randperm(total, generator=g)
    table = torch.full((len(lens), max(per) + 1), -7, dtype=torch.int32)
    at = 0
    for i, p in enumerate(per):
        table[i, :p] = order[at:at + p]
        at += p
    return cache, table


def offsets(n):
    return torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)


def assert_cache(cache, ref, table, lens, what=""):
    for side, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        got = RefCache(cache)
        for i, n in enumerate(lens):
            if n == 0:
                continue
            a, b = got.values(side, table[i], 0, n), ref.values(side, table[i], 0, n)
            at = torch.arange(n)
            pg = table[i][at // cache.page_size].long()
            step = ref.scale[side][pg, :, at % cache.page_size // cache.block][..., None]
            err = (a - b).abs()
            assert (err <= step * 1.001).all(), f"{what} side {side} seq {i}"
            off = (err > step * 127 * 2.0 ** -18).double().mean()
            assert off <= 1e-3, f"{what} side {side} seq {i}: {float(off)} of the values differ"


@gpu
@pytest.mark.parametrize("H,D,page,block,dt,rot,inter,norm", [
    (2, 128, 64, 16, torch.float32, 128, False, True),
    (1, 64, 16, 16, torch.bfloat16, 64, True, False),
    (3, 64, 96, 32, torch.float16, 32, False, True),
    (2, 256, 64, 64, torch.float32, 256, False, True),
    (8, 128, 32, 32, torch.bfloat16, 64, True, True),
    (1, 256, 32, 16, torch.float16, 0, False, False),
    (2, 64, 128, 64, torch.float32, 64, False, True),
    (5, 128, 64, 64, torch.float16, 128, False, False),
])
def test_append_steps(H, D, page, block, dt, rot, inter, norm):
    """Several appends in turn: ragged prompts, single tokens, an empty sequence, ends inside blocks and pages."""
    g = torch.Generator().manual_seed(H * D + block)
    steps = [[37, 1, 0, block, 5], [1, 1, 1, 1, 1], [3, 0, 70, 1, block - 5], [1, 1, 1, 1, 1]]
    final = [sum(x) for x in zip(*steps)]
    cache, table = make_cache(g, final, H, D, page, block, fill=False)
    ref = RefCache(cache)
    for side in (0, 1):
        ref.scale[side].zero_()
    cos, sin = rotary_tables(200, rot) if rot else (None, None)
    w = 1 + 0.2 * torch.randn(D, generator=g) if norm else None
    wq = 1 + 0.2 * torch.randn(D, generator=g) if norm else None
    dev = [t.cuda() if t is not None else None for t in (cos, sin, w, wq)]
    lens = [0] * 5
    G = 3
    for step, n in enumerate(steps):
        total = sum(n)
        rows = (torch.randn(total, (G + 2) * H, D, generator=g) * torch.rand(total, 1, 1, generator=g) * 3).to(dt)
        lens = [a + b for a, b in zip(lens, n)]
        cu = offsets(n)
        r = rows.cuda()
        q, k, v = r[:, :G * H], r[:, G * H:(G + 1) * H], r[:, (G + 1) * H:]
        each = step in (1, 3)                                 # one token each: with and without offsets
        qo = api.kv_append(cache, k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           None if step == 1 and each else cu.cuda(), dev[0], dev[1], inter, dev[2], 1e-5,
                           q if step != 2 else None, dev[3], q_dtype=torch.float32)
        for i in range(5):
            start = lens[i] - n[i]
            part = rows[cu[i]:cu[i + 1]]
            kk = [ref_norm_rope(part[j, G * H:(G + 1) * H], w, 1e-5, cos[start + j] if rot else None,
                                sin[start + j] if rot else None, inter) for j in range(n[i])]
            if n[i]:
                ref.append(0, table[i], start, torch.stack(kk))
                ref.append(1, table[i], start, part[:, (G + 1) * H:])
            if step != 2:
                for j in range(n[i]):
                    qr = ref_norm_rope(part[j, :G * H], wq, 1e-5, cos[start + j] if rot else None,
                                       sin[start + j] if rot else None, inter)
                    assert_close(qo[cu[i] + j], qr, 20 * 2.0 ** -24 * qr.abs().amax(-1, keepdim=True) + 1e-7, "q")
        assert_cache(cache, ref, table, lens, f"step {step}")
        # later steps start from the same codes, so that one-step differences do not add up
        ref = RefCache(cache)
    assert api.read_device_errors() == 0


@gpu
def test_append_grows_the_scale_and_rescales_held_codes():
    cache, table = make_cache(torch.Generator().manual_seed(1), [40], 1, 64, 64, 16, fill=False)
    tb = table.cuda()
    small = torch.full((3, 1, 64), 0.5, device="cuda")
    small[:, :, ::2] = -0.25
    api.kv_append(cache, small, small, tb, torch.tensor([3], dtype=torch.int32, device="cuda"),
                  torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    pg = int(table[0, 0])
    assert cache.k_scale[pg, 0, 0].item() == np.float32(0.5) / np.float32(127)
    big = torch.full((1, 1, 64), -2.0, device="cuda")
    api.kv_append(cache, big, small[:1], tb, torch.tensor([4], dtype=torch.int32, device="cuda"))
    assert cache.k_scale[pg, 0, 0].item() == np.float32(2) / np.float32(127)
    assert cache.k[pg, 0, 3].tolist() == [-127] * 64
    assert cache.k[pg, 0, 0, :2].tolist() == [-16, 32]        # -64 / 4, 127 / 4 rounded
    assert cache.v_scale[pg, 0, 0].item() == np.float32(0.5) / np.float32(127)
    assert cache.v[pg, 0, 3, :2].tolist() == [-64, 127]


@gpu
def test_append_zero_tiny_and_huge_values():
    cache, table = make_cache(torch.Generator().manual_seed(1), [48], 1, 64, 16, 16, fill=False)
    x = torch.zeros(48, 1, 64, device="cuda")
    x[16:32] = 1e-30                                          # scale below 2^-63: stored as zeros
    x[32:] = torch.linspace(-1, 1, 64, device="cuda") * 3e38
    lens = torch.tensor([48], dtype=torch.int32, device="cuda")
    api.kv_append(cache, x, x, table.cuda(), lens, torch.tensor([0, 48], dtype=torch.int32, device="cuda"))
    k, v = api.kv_read(cache, table.cuda(), lens, 48, torch.tensor([0, 48], dtype=torch.int32, device="cuda"),
                       torch.float32)
    assert (k[:32] == 0).all() and torch.equal(k, v)
    assert torch.isfinite(k).all() and ((k[32:] - x[32:]).abs() <= 3e38 / 127 * 0.51).all()


@gpu
def test_append_flags_and_skips_what_does_not_fit():
    g = torch.Generator().manual_seed(3)
    cache, table = make_cache(g, [32, 32], 2, 64, 16, 16)
    x = torch.randn(6, 2, 64, generator=g).cuda()
    cu = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    bad = table.clone()
    bad[0, 1] = cache.pages                                   # outside the cache
    before = cache.k.clone()
    api.read_device_errors()
    api.kv_append(cache, x, x, bad.cuda(), torch.tensor([30, 20], dtype=torch.int32, device="cuda"), cu)
    assert api.read_device_errors() == api.DEVERR_PAGE
    changed = (cache.k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(table[1, 1])]
    # longer than its table: the first sequence's last token has no place
    api.kv_append(cache, x, x, table[:, :2].contiguous().cuda(), torch.tensor([33, 20], dtype=torch.int32, device="cuda"),
                  cu)
    assert api.read_device_errors() == api.DEVERR_LENGTH
    # positions past the rotation table
    cos, sin = (t.cuda() for t in rotary_tables(19, 64))
    api.kv_append(cache, x, x, table.cuda(), torch.tensor([10, 20], dtype=torch.int32, device="cuda"), cu, cos, sin)
    assert api.read_device_errors() == api.DEVERR_POSITION


@gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,D,page,block", [(3, 64, 48, 16), (1, 128, 64, 64), (2, 256, 32, 32)])
def test_read(dt, H, D, page, block):
    g = torch.Generator().manual_seed(7)
    lens, n = [100, 1, 33, 64, 7], [100, 1, 5, 0, 3]
    cache, table = make_cache(g, lens, H, D, page, block)
    cu = offsets(n)
    k, v = api.kv_read(cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), sum(n), cu.cuda(), dt)
    ref = RefCache(cache)
    for i in range(5):
        for side, x in enumerate((k, v)):
            want = ref.values(side, table[i], lens[i] - n[i], lens[i])
            assert torch.equal(x[cu[i]:cu[i + 1]].cpu(), want.float().to(dt))
    assert api.read_device_errors() == 0


@gpu
def test_read_rows_without_a_place_are_zeros():
    g = torch.Generator().manual_seed(7)
    cache, table = make_cache(g, [20, 20], 1, 64, 16, 16)
    table[1, 0] = -1
    k, v = api.kv_read(cache, table.cuda(), torch.tensor([2, 20], dtype=torch.int32, device="cuda"), 24,
                       torch.tensor([0, 4, 24], dtype=torch.int32, device="cuda"), torch.float32)
    assert (k[:2] == 0).all() and (k[2:4] != 0).any() and (k[4:20] == 0).all() and (v[20:] != 0).any()
    assert api.read_device_errors() == api.DEVERR_LENGTH | api.DEVERR_PAGE


# ------------------------------------------------------------------------------------------------ attention
def ref_attention(q, cache, table, lens, n, scale, causal, window):
    ref = RefCache(cache)
    T, Hq, D = q.shape
    group = Hq // cache.kv_heads
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    vmax = 0.0
    at = 0
    for i, (L, m) in enumerate(zip(lens, n)):
        if m and L:
            k, v = (ref.values(side, table[i], 0, L) for side in (0, 1))
            vmax = max(vmax, float(v.abs().max()))
            place = torch.arange(L - m, L)[:, None]
            j = torch.arange(L)[None]
            see = torch.ones(m, L, dtype=torch.bool)
            if causal:
                see = j <= place
                if window:
                    see &= j > place - window
            for h in range(Hq):
                s = (q[at:at + m, h].double() @ k[:, h // group].T * scale).masked_fill(~see, -math.inf)
                top = s.amax(-1, keepdim=True)
                p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
                z = p.sum(-1, keepdim=True)
                out[at:at + m, h] = (p / torch.where(z > 0, z, torch.ones_like(z))) @ v[:, h // group]
                lse[at:at + m, h] = (torch.log(z) + top)[:, 0]
        at += m
    return out, lse, vmax


def check_attention(lens, n, Hq, H, D, page, block, qt=torch.bfloat16, ot=torch.float32, causal=True, window=0,
                    scale=None, seed=0, spread=1.0, tamper=None, **more):
    g = torch.Generator().manual_seed(seed + sum(lens) + D)
    cache, table = make_cache(g, lens, H, D, page, block)
    q = (torch.randn(sum(n), Hq, D, generator=g) * spread).to(qt)
    if tamper:
        tamper(cache, table, q)
    scale = D ** -0.5 if scale is None else scale
    want, wlse, vmax = ref_attention(q, cache, table, lens, n, scale, causal, window)
    api.read_device_errors()
    cu = None if more.pop("no_cu", False) else offsets(n).cuda()
    out, lse = api.attention(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             max_kv_len=more.pop("max_kv_len", max(lens)), cu_tokens=cu,
                             max_tokens=more.pop("max_tokens", max(n)), scale=scale, causal=causal, window=window,
                             out_dtype=ot, return_lse=True, **more)
    tol = vmax * (2.0 ** -11 + 2.0 ** -16 + ULP[ot])
    assert_close(out, want, torch.full_like(want, tol), "out")
    empty = wlse == -math.inf
    assert torch.equal(torch.isneginf(lse).cpu(), empty)
    assert (out.cpu()[empty] == 0).all()
    err = (lse.double().cpu() - wlse)[~empty].abs()
    assert (err <= 2.0 ** -18 + 2.0 ** -20 * wlse[~empty].abs()).all(), float(err.max())
    assert api.read_device_errors() == 0
    return out


SHAPES = [(4, 4, 64, 16, 16), (8, 2, 128, 64, 16), (7, 1, 128, 32, 32), (16, 1, 64, 64, 64), (6, 2, 256, 48, 16),
          (10, 2, 256, 64, 64), (20, 1, 128, 128, 32)]


@gpu
@pytest.mark.parametrize("Hq,H,D,page,block", SHAPES)
@pytest.mark.parametrize("lens", [[1, 2, 15, 16, 17], [31, 64, 65, 127, 128], [600, 3, 1025, 300, 129]])
def test_attention_single_tokens(Hq, H, D, page, block, lens):
    check_attention(lens, [1] * 5, Hq, H, D, page, block, no_cu=lens[0] == 31)


@gpu
@pytest.mark.parametrize("Hq,H,D,page,block", SHAPES)
@pytest.mark.parametrize("lens,n", [([5, 40, 333], [5, 2, 3]), ([70, 0, 130], [65, 0, 17]), ([300, 129, 1], [128, 129, 1]),
                                    ([257, 900], [257, 131])])
def test_attention_prompts(Hq, H, D, page, block, lens, n):
    check_attention(lens, n, Hq, H, D, page, block, torch.float16 if D == 64 else torch.bfloat16)


@gpu
@pytest.mark.parametrize("window", [1, 7, 16, 100, 5000])
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 3, 150], [300, 150, 1]])
def test_attention_window(window, n):
    check_attention([400, 150, 33], n, 8, 2, 128, 32, 16, window=window)
    check_attention([400, 150, 33], n, 6, 2, 64, 64, 64, window=window)


@gpu
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 3, 33], [300, 150, 33]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_without_causal_mask(n, D):
    check_attention([400, 150, 33], n, 8, 2, D, 32, 16, causal=False)


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,n", [([0, 5], [1, 1]), ([0, 3, 9], [4, 7, 9]), ([2, 0, 100], [200, 150, 130])])
def test_attention_rows_that_see_nothing(lens, n, D):
    """Sequences shorter than their new tokens: the first rows see no position."""
    check_attention(lens, n, 8, 2, D, 32, 16)
    check_attention(lens, n, 8, 2, D, 32, 16, causal=False)


@gpu
@pytest.mark.parametrize("qt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ot", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [[1, 1], [130, 20]])
def test_attention_types(qt, ot, n):
    check_attention([200, 77], n, 8, 4, 128, 64, 32, qt, ot)


@gpu
@pytest.mark.parametrize("n", [[1, 1, 1], [9, 140, 40]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_split_along_the_cache(n, D):
    """Long caches of few rows are cut in parts and joined; parts that a row does not see at all among them."""
    check_attention([5000, 150, 2311], n, 4, 1, D, 64, 16)
    check_attention([5000, 150, 2311], n, 4, 1, D, 64, 64, window=700)


@gpu
@pytest.mark.parametrize("n", [[1, 1], [3, 150]])
def test_attention_sharp_rows_and_scales(n):
    """Scores far apart, queries of extreme bf16 magnitude, zero value blocks, scales of many magnitudes."""
    def tamper(cache, table, q):
        q[0] *= 8.0
        cache.v_scale[int(table[0, 0]), :, 0] = 0
        cache.v[int(table[0, 0]), :, :16] = 0
        cache.v_scale[int(table[0, 2])] = 1e-7
        cache.k_scale[int(table[1, 0]), :, 0] = 0
    check_attention([300, 200], n, 8, 2, 128, 64, 16, tamper=tamper)

    def tiny(cache, table, q):
        q *= 2.0 ** -100
        cache.v_scale.mul_(2.0 ** -30)
    check_attention([300, 200], n, 8, 2, 64, 64, 16, tamper=tiny, scale=2.0 ** 97)
    check_attention([300, 200], n, 8, 2, 64, 64, 16, scale=-0.1)
    check_attention([300, 200], n, 8, 2, 256, 64, 16, scale=0.0)


@gpu
@pytest.mark.parametrize("n", [[1, 1], [3, 150]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_ignores_what_lies_past_the_length(n, D):
    """NaN scales and any codes in blocks and pages past the length, and invalid table entries, change nothing."""
    g = torch.Generator().manual_seed(5)
    lens = [290, 163]
    cache, table = make_cache(g, lens, 2, D, 64, 16)
    q = torch.randn(sum(n), 8, D, generator=g).bfloat16().cuda()
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = api.attention(q, cache, table.cuda(), kv, max(lens), offsets(n).cuda(), max(n))
    used = torch.zeros(cache.pages, 64, dtype=torch.bool)
    for i, L in enumerate(lens):
        at = torch.arange(L)
        used[table[i][at // 64].long(), at % 64] = True
    dead = (~used).cuda()
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.permute(0, 2, 1, 3)[dead] = -128
        s.permute(0, 2, 1)[dead.view(cache.pages, 4, 16).all(-1)] = float("nan")
    table[:, -1] = 2 ** 30
    again = api.attention(q, cache, table.cuda(), kv, max(lens), offsets(n).cuda(), max(n))
    assert torch.equal(first, again)
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("n", [1, 140])
def test_attention_strided_rows_streams_and_workspace(n):
    """Queries and outputs that are slices of wider rows, another stream, a caller's workspace: the same bits."""
    g = torch.Generator().manual_seed(11)
    lens = [3000, 2900]
    cache, table = make_cache(g, lens, 2, 128, 64, 32)
    wide = torch.randn(2 * n, 13, 128, generator=g).bfloat16().cuda()
    q = wide[:, 2:10]
    kv, cu, tb = torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets([n, n]).cuda(), table.cuda()
    want = api.attention(q.contiguous(), cache, tb, kv, 3000, cu, n)
    need = api.attention_workspace_bytes(2 * n, 8, 2, 128, 2, n, 3000)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((2 * n, 12, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    api.attention(q, cache, tb, kv, 3000, cu, n, out=out[:, 1:9], workspace=ws, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out[:, 1:9], want)
    assert (out[:, 0] == 5).all() and (out[:, 9:] == 5).all() and (ws[need:] == 0xFF).all()


@gpu
@pytest.mark.parametrize("n", [1, 140])
def test_attention_flags_lengths_and_pages(n):
    g = torch.Generator().manual_seed(2)
    cache, table = make_cache(g, [300], 1, 64, 64, 16)
    q = torch.randn(n, 4, 64, generator=g).bfloat16().cuda()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kv = torch.tensor([300], dtype=torch.int32, device="cuda")
    api.read_device_errors()
    api.attention(q, cache, table.cuda(), kv, 200, cu, n)
    assert api.read_device_errors() == api.DEVERR_LENGTH
    table[0, 1] = -5
    out = api.attention(q, cache, table.cuda(), kv, 300, cu, n)
    assert api.read_device_errors() == api.DEVERR_PAGE and torch.isfinite(out.float()).all()


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,n,Hq,H", [([9001, 300], [1, 1], 4, 1),                  # 71 parts of 128
                                         ([5000, 77, 4999], [3, 1, 4], 4, 1),          # 40 parts, several rows
                                         ([20011, 1025, 1024, 30], [1] * 4, 8, 8),     # parts of 1024
                                         ([700, 33, 385, 384] * 10, [1] * 40, 64, 8)])  # more rows than resident blocks
def test_attention_joins(lens, n, Hq, H, D):
    """Every form of the join: few rows of many parts, of a few, and many rows; sequences of one part among them."""
    check_attention(lens, n, Hq, H, D, 64, 16)


@gpu
@pytest.mark.parametrize("n", [1, 33])
def test_attention_offsets_past_32_bits(n):
    """A cache whose codes take more than 2^32 bytes, with the sequence in its last pages."""
    pages = (1 << 32) // (64 * 128) + 40
    cache = api.KVCache.empty(pages, 1, 128, 64, 16)
    L = 500
    table = torch.arange(pages - 8, pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y = (torch.randn(L, 1, 128, device="cuda", generator=g) for _ in range(2))
    kv, cu = torch.tensor([L], dtype=torch.int32, device="cuda"), torch.tensor([0, L], dtype=torch.int32, device="cuda")
    api.kv_append(cache, x, y, table, kv, cu)
    k, v = api.kv_read(cache, table, kv, L, cu, torch.float32)
    assert (k - x).abs().max() <= 6 / 127 and (v - y).abs().max() <= 6 / 127
    q = torch.randn(n, 4, 128, device="cuda", generator=g).half()
    out = api.attention(q, cache, table, kv, L, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n,
                        out_dtype=torch.float32)
    s = torch.einsum("qhd,kd->qhk", q.double(), k[:, 0].double()) * 128 ** -0.5
    s.masked_fill_(torch.arange(L, device="cuda") > torch.arange(L - n, L, device="cuda")[:, None, None], -math.inf)
    want = (torch.softmax(s, -1) @ v[:, 0].double()).cpu()
    assert_close(out, want, torch.full_like(want, float(v.abs().max()) * (2.0 ** -11 + 2.0 ** -16)))


@gpu
def test_steps_in_a_graph():
    """Append and attention captured once and replayed with growing lengths (device-side lengths only)."""
    g = torch.Generator().manual_seed(4)
    H, Hq, D, n_seq = 2, 8, 128, 3
    cache, table = make_cache(g, [200] * n_seq, H, D, 64, 16, fill=False)
    tb = table.cuda()
    cos, sin = (t.cuda() for t in rotary_tables(256, D))
    rows = torch.zeros(n_seq, Hq + 2 * H, D, device="cuda")
    lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    q = torch.empty(n_seq, Hq, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(n_seq, Hq, D, device="cuda")
    ws = torch.empty(api.attention_workspace_bytes(n_seq, Hq, H, D, n_seq, 1, 200) + 16, dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        api.kv_append(cache, rows[:, Hq:Hq + H], rows[:, Hq + H:], tb, lens, None, cos, sin, q=rows[:, :Hq], q_out=q)
        api.attention(q, cache, tb, lens, 200, out=out, workspace=ws)

    step()
    lens.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens.zero_()
    for i in range(40):
        rows.copy_(torch.randn(rows.shape, generator=g))
        graph.replay()
    assert lens.tolist() == [40] * n_seq
    want, _, vmax = ref_attention(q.cpu(), cache, table, [40] * n_seq, [1] * n_seq, D ** -0.5, True, 0)
    assert_close(out, want, torch.full_like(want, vmax * (2.0 ** -11 + 2.0 ** -16)))
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_prompt_among_single_tokens(D):
    """One prompt and many single tokens in a batch, in every order: rows of many sequences in one launch."""
    n = [1, 1, 300, 1, 0, 1, 17, 1, 1, 1] + [1] * 30
    lens = [90, 1, 300, 33, 5, 64, 40, 128, 700, 16] + [20 + i for i in range(30)]
    check_attention(lens, n, 8, 2, D, 64, 16)
    check_attention(lens[::-1], n[::-1], 6, 1, D, 32, 32, window=50)
