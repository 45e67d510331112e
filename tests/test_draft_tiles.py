"""Attention of a tree's rows in the kernel that shares out tiles (csrc/attn_tree.cu), at sizes that the rule of csrc/attn_api.cu
sends there, which is asserted: batches of which a block has more tiles than it lists at once, and calls that repeat.
References and tolerances as in test_draft_tree.py."""
import ctypes
import math

import pytest
import torch

import test_draft_tree as T
from test_attention_ops import ULP, assert_close, offsets

from block_quantized_int8_q8_gb300 import _build, api

gpu = pytest.mark.gpu
FEW, TILES, TILED = range(3)                                  # TreeKernel of csrc/attn.h
TILE, SHARES, LISTED = 128, 152, 256                          # tokens of a tile, blocks, tiles that a block lists at once


def kernel(group, kv_heads, dim, seqs, most, max_kv):
    _build.build()
    f = getattr(api.load(), "_ZN3mmq11tree_kernelEiiiixx")
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64] * 2
    f.restype = ctypes.c_int
    return f(group, kv_heads, dim, seqs, most, max_kv)


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
