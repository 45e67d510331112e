"""Sizes just past those from which the operators work in another form, with odd remainders: more sequences than the threads
that look for one, more tokens a block, smaller blocks for long reads (tolerances as in test_attention_ops.py; the cache
to the bit)."""
import pytest
import torch

from test_attention_ops import RefCache, ULP, assert_close, check_attention, make_cache, offsets, rotary_tables

from block_quantized_int8_q8_gb300 import api

gpu = pytest.mark.gpu


def ref_heads(x, w, eps, cos, sin, interleaved):
    """Norm and rotation of x [T, H, D] in 64 bits; cos, sin [T, rot/2] of each token's position."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    half = cos.shape[1]
    at = torch.arange(half)
    a, b = (2 * at, 2 * at + 1) if interleaved else (at, at + half)
    c, s = cos.double()[:, None], sin.double()[:, None]
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


class ExactCache(RefCache):
    """The cache's format to the bit: quotients and the product of the rescale in f32, as it is defined."""

    def append(self, side, row, start, x):
        c, s, B, P = self.codes[side], self.scale[side], self.c.block, self.c.page_size
        n = x.shape[0]
        for b in range(start // B * B, start + n, B):
            pg, off = int(row[b // P]), b % P
            lo, hi = max(start, b), min(start + n, b + B)
            new = x[lo - start:hi - start].float().transpose(0, 1)
            need = new.abs().amax((1, 2)) / 127
            need[need < 2.0 ** -63] = 0
            old = torch.zeros_like(need) if lo == b else s[pg, :, off // B].float()
            d = torch.maximum(old, need)
            safe = torch.where(d > 0, d, torch.ones_like(d))[:, None, None]
            if lo > b:
                held = c[pg, :, off:off + lo - b].float()
                c[pg, :, off:off + lo - b] = torch.round(held * (old[:, None, None] / safe)).double()
            c[pg, :, off + lo - b:off + hi - b] = torch.round(new / safe).clamp(-127, 127).double()
            s[pg, :, off // B] = d.double()


def lengths(seqs, most, g, empty=7):
    """Ragged numbers, every empty-th one zero."""
    n = torch.randint(1, most + 1, (seqs,), generator=g)
    n[::empty] = 0
    return n.tolist()


@gpu
@pytest.mark.parametrize("tokens", [607, 609, 1217, 1823])
@pytest.mark.parametrize("D,hq,hk,rot,inter,it,ot", [(128, 5, 2, 128, False, torch.bfloat16, torch.bfloat16),
                                                     (64, 9, 3, 32, True, torch.float32, torch.float16),
                                                     (256, 3, 1, 256, False, torch.float16, torch.float32)])
def test_norm_rope_of_several_tokens_a_block(tokens, D, hq, hk, rot, inter, it, ot):
    g = torch.Generator().manual_seed(tokens)
    rows = (torch.randn(tokens, hq + hk, D, generator=g) * 2).to(it)
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g) for _ in range(2))
    cos, sin = rotary_tables(500, rot)
    pos = torch.randint(0, 500, (tokens,), generator=g, dtype=torch.int32)
    dev = rows.cuda()
    outs = api.qk_norm_rope(dev[:, :hq], dev[:, hq:], pos.cuda(), cos.cuda(), sin.cuda(), wq.cuda(), wk.cuda(), 1e-6, inter,
                            dtype=ot)
    for x, o, w in ((rows[:, :hq], outs[0], wq), (rows[:, hq:], outs[1], wk)):
        ref = ref_heads(x, w, 1e-6, cos[pos.long()], sin[pos.long()], inter)
        assert_close(o, ref, 16 * 2.0 ** -24 * ref.abs().amax(-1, keepdim=True) + ULP[ot] * ref.abs() + 1e-7)
    assert api.read_device_errors() == 0


def append_and_compare(n, before, H, G, D, page, block, seed):
    """Append n[i] tokens to sequences of before[i].  Keys and values as they are, so that the cache is known to the bit; the
    queries normed and rotated."""
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(n, before)]
    cache, table = make_cache(g, lens, H, D, page, block)
    ref = ExactCache(cache)
    cos, sin = rotary_tables(max(lens), D)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    total = sum(n)
    rows = torch.randn(total, (G + 2) * H, D, generator=g) * 2
    r = rows.cuda()
    q, k, v = (rows[:, a:b] for a, b in ((0, G * H), (G * H, (G + 1) * H), ((G + 1) * H, (G + 2) * H)))
    tb, kv, cu = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets(n)
    pos = torch.cat([torch.arange(L - m, L) for L, m in zip(lens, n)])
    api.kv_append(cache, r[:, G * H:(G + 1) * H], r[:, (G + 1) * H:], tb, kv, cu.cuda())
    for i, (m, b) in enumerate(zip(n, before)):
        if m:
            ref.append(0, table[i], b, k[cu[i]:cu[i + 1]])
            ref.append(1, table[i], b, v[cu[i]:cu[i + 1]])
    got = RefCache(cache)
    for side in (0, 1):
        assert torch.equal(got.codes[side], ref.codes[side]) and torch.equal(got.scale[side], ref.scale[side])
    back = api.kv_read(cache, tb, kv, total, cu.cuda(), torch.float32)
    for side in (0, 1):
        want = torch.cat([got.values(side, table[i], L - m, L) for i, (L, m) in enumerate(zip(lens, n)) if m])
        assert torch.equal(back[side].cpu(), want.float())
    # the same rows again with the queries, keys rotated: each sequence's last tokens anew
    qo = api.kv_append(cache, r[:, G * H:(G + 1) * H], r[:, (G + 1) * H:], tb, kv, cu.cuda(), cos.cuda(), sin.cuda(), False,
                       None, 1e-5, r[:, :G * H], w.cuda(), q_dtype=torch.float32)
    qr = ref_heads(q, w, 1e-5, cos[pos], sin[pos], False)
    assert_close(qo, qr, 20 * 2.0 ** -24 * qr.abs().amax(-1, keepdim=True) + 1e-7, "q")
    assert api.read_device_errors() == 0


# blocks of 128, 256 and 512 threads look for a sequence, in slots by tokens (few new ones) and by blocks
@gpu
@pytest.mark.parametrize("seqs", [129, 300, 700])
@pytest.mark.parametrize("D,page,block", [(64, 32, 16), (128, 64, 32), (128, 64, 64)])
@pytest.mark.parametrize("most", [1, 40])
def test_append_and_read_of_many_sequences(seqs, D, page, block, most):
    g = torch.Generator().manual_seed(seqs + most)
    n = lengths(seqs, most, g)
    append_and_compare(n, torch.randint(0, 70, (seqs,), generator=g).tolist(), 1, 2, D, page, block, seqs)


# four tokens of queries a block: a block of several sequences, of a sequence's end and the next, and a short last one
@gpu
@pytest.mark.parametrize("n", [[1217], [1499], [3, 0, 600, 1, 1, 0, 2, 611], [2] * 609 + [1], [1] * 1218])
@pytest.mark.parametrize("D", [64, 256])
def test_append_of_several_tokens_of_queries_a_block(n, D):
    append_and_compare(n, [(5 * i) % 23 for i in range(len(n))], 2, 3, D, 64, 16, len(n))


@gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,D", [(1, 64), (3, 128), (2, 256)])
@pytest.mark.parametrize("tokens", [32768, 32769])
def test_long_reads(dt, H, D, tokens):
    g = torch.Generator().manual_seed(D)
    n = [20001, 0, 1, tokens - 20001 - 1 - 77, 77]
    lens = [20100, 5, 1, tokens - 20001 - 1 - 77, 300]
    cache, table = make_cache(g, lens, H, D, 64, 16)
    cu = offsets(n)
    k, v = api.kv_read(cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), tokens, cu.cuda(), dt)
    ref = RefCache(cache)
    for i in range(len(n)):
        for side, x in enumerate((k, v)):
            want = ref.values(side, table[i], lens[i] - n[i], lens[i])
            assert torch.equal(x[cu[i]:cu[i + 1]].cpu(), want.float().to(dt))
    assert api.read_device_errors() == 0


# one sequence long enough to be cut in parts, so that every row goes through the join's search
@gpu
@pytest.mark.parametrize("seqs", [129, 300, 700])
@pytest.mark.parametrize("Hq,H,D", [(2, 1, 64), (2, 2, 128), (3, 1, 256)])
def test_single_tokens_of_many_sequences(seqs, Hq, H, D):
    g = torch.Generator().manual_seed(seqs)
    n = [min(x, 1) for x in lengths(seqs, 2, g)]
    lens = torch.randint(1, 90, (seqs,), generator=g).tolist()
    lens[seqs // 2], n[seqs // 2] = 3001, 1
    lens[-1], n[-1] = 2500, 2
    check_attention(lens, n, Hq, H, D, 64, 16)


@gpu
@pytest.mark.parametrize("seqs", [129, 300, 700])
@pytest.mark.parametrize("Hq,H,D", [(2, 1, 64), (2, 2, 128), (1, 1, 256)])
def test_prompts_of_many_sequences(seqs, Hq, H, D):
    """Row blocks numbered through the packed rows: one long prompt among many short ones."""
    g = torch.Generator().manual_seed(seqs)
    n = lengths(seqs, 5, g)
    n[seqs // 3] = 700
    lens = [m + int(x) for m, x in zip(n, torch.randint(0, 60, (seqs,), generator=g))]
    check_attention(lens, n, Hq, H, D, 64, 16)
    check_attention(lens[::-1], n[::-1], Hq, H, D, 32, 32, window=33)
