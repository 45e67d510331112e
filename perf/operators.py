"""Cases and plain forms of the attention operators over the 8-bit paged key/value cache.

Four operators of a serving step, between the fused q/k/v projection and the output projection:

  norm_rope   RMS norm of each query and key head (learned weight) and the position rotation, one pass
  append      norm and rotation of new keys (and queries), then keys and values quantized into the paged cache
  read        a range of each sequence's cache turned back into floating-point rows
  attention   softmax(q k^T) v over the cache, for single new tokens and for whole prompts

The cache holds int8 codes [pages, kv heads, page size, head dim] and one f32 scale for each block of `block`
tokens and head: value = scale * code, scale = amax / 127, code = round-half-even(value / scale).  An append into
a partly filled block keeps the block's scale unless a new value needs a larger one; then the codes that are
already there are rescaled to it.  A block whose first token is appended starts afresh.
"""
import math

import torch

own = False

#: a block scale below this is stored as zero (all codes zero)
TINY = 2.0 ** -63
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a few sequences' new token, straight from the f32 output of the quantized projection: latency counts
        {"name": "norm_rope_4_tokens", "op": "norm_rope", "tokens": 4, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "dtype": "f32"},
        # a long prompt chunk: bandwidth
        {"name": "norm_rope_8191_tokens", "op": "norm_rope", "tokens": 8191, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "dtype": "bf16"},
        # one decode step of a batch: one token for each of 64 sequences, queries and keys normed and rotated
        {"name": "append_decode_64", "op": "append", "seqs": 64, "new": 1, "past": 700, "ragged": True, "heads": 32,
         "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "norm": True, "page": 64, "block": 16,
         "dtype": "f32"},
        # prompts of five requests, partial rotation in adjacent pairs, no norm, after what is already cached
        {"name": "append_prefill_5x2047", "op": "append", "seqs": 5, "new": 2047, "past": 333, "ragged": True,
         "heads": 32, "kv_heads": 8, "dim": 128, "rot": 64, "interleaved": True, "norm": False, "page": 32,
         "block": 32, "dtype": "bf16"},
        # the last tokens of a few requests, as a host-side check or a migration of a request reads them
        {"name": "read_3x500", "op": "read", "seqs": 3, "new": 500, "past": 41, "ragged": True, "kv_heads": 8,
         "dim": 128, "page": 16, "block": 16, "dtype": "f32"},
        # whole prefixes turned back into 16-bit rows
        {"name": "read_8x16384", "op": "read", "seqs": 8, "new": 16384, "past": 0, "ragged": False, "kv_heads": 8,
         "dim": 128, "page": 64, "block": 64, "dtype": "bf16"},
        # the first tokens of a chat: one sequence, a short cache, nothing but latency
        {"name": "decode_1x77", "op": "attention", "seqs": 1, "new": 1, "past": 76, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "causal": True, "window": 0, "page": 16, "block": 16, "dtype": "bf16"},
        # a full serving batch with ragged contexts: bandwidth of the cache
        {"name": "decode_64x8192", "op": "attention", "seqs": 64, "new": 1, "past": 8191, "ragged": True, "heads": 32,
         "kv_heads": 8, "dim": 128, "causal": True, "window": 0, "page": 64, "block": 16, "dtype": "bf16"},
        # one request with a very long document: few rows, the work split along the cache
        {"name": "decode_1x131072", "op": "attention", "seqs": 1, "new": 1, "past": 131001, "ragged": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "causal": True, "window": 0, "page": 64, "block": 64,
         "dtype": "bf16"},
        # every head with a cache of its own and small heads, four draft tokens checked at once
        {"name": "verify_16x4_mha64", "op": "attention", "seqs": 16, "new": 4, "past": 2000, "ragged": True,
         "heads": 32, "kv_heads": 32, "dim": 64, "causal": True, "window": 0, "page": 32, "block": 32,
         "dtype": "f16"},
        # prompts of four requests at once: matrix products
        {"name": "prefill_4x4096", "op": "attention", "seqs": 4, "new": 4096, "past": 0, "ragged": True, "heads": 32,
         "kv_heads": 8, "dim": 128, "causal": True, "window": 0, "page": 64, "block": 16, "dtype": "bf16"},
        # a chunk of a long document against what is already cached
        {"name": "chunk_2048_after_30000", "op": "attention", "seqs": 1, "new": 2048, "past": 30001, "ragged": False,
         "heads": 16, "kv_heads": 2, "dim": 128, "causal": True, "window": 0, "page": 64, "block": 32,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "append", "read", "attention", "attention", "attention", "attention"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 8, 16])
    heads = kv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64) if b <= page])
    if op == "norm_rope":
        return {"op": op, "tokens": _log(rng, 1, 8191), "heads": heads, "kv_heads": kv, "dim": dim,
                "rot": rng.choice([dim, dim // 2]), "interleaved": rng.random() < 0.4,
                "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op in ("append", "read"):
        seqs = _log(rng, 1, 64)
        new = 1 if op == "append" and rng.random() < 0.5 else _log(rng, 1, 16384 // seqs)
        c = {"op": op, "seqs": seqs, "new": new, "past": _log(rng, 1, 2000), "ragged": rng.random() < 0.7}
        if op == "append":
            c.update({"heads": heads, "rot": rng.choice([dim, dim // 2]), "interleaved": rng.random() < 0.4,
                      "norm": rng.random() < 0.5})
        c.update({"kv_heads": kv, "dim": dim, "page": page, "block": block,
                  "dtype": rng.choice(["f32", "bf16", "f16"])})
        return c
    c = {"op": op, "ragged": rng.random() < 0.7, "heads": heads, "kv_heads": kv, "dim": dim, "causal": True,
         "window": 0, "page": page, "block": block, "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if rng.random() < 0.5:                     # one or a few new tokens over a cache of up to 2**21 rows in all
        c["seqs"] = _log(rng, 1, 64)
        c["new"] = rng.choice([1, 1, 1, 2, 5])
        c["past"] = _log(rng, 8, min(262144, (1 << 21) // (c["seqs"] * kv)))
    else:                                      # prompts and chunks: up to 2**30 score entries in all
        c["seqs"] = _log(rng, 1, 8)
        most = (1 << 30) // (c["seqs"] * heads)
        c["new"] = _log(rng, 17, min(4096, math.isqrt(most)))
        c["past"] = _log(rng, 1, max(2, min(32768, most // c["new"] - c["new"])))
        c["causal"] = rng.random() < 0.85
    if c["causal"] and rng.random() < 0.25:
        c["window"] = _log(rng, 16, 4096)
    return c


def _sizes(case):
    """New tokens and cache lengths (after them) of every sequence: odd and ragged, from the case alone."""
    n = case["seqs"]
    new, past = [], []
    for i in range(n):
        f = 1.0 if not case["ragged"] or i == 0 else ((i * 2654435761) % 1000 + 1) / 1000.0
        new.append(max(1, int(case["new"] * (0.25 + 0.75 * f))))
        past.append(int(case["past"] * f))
    return new, past


# ------------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rotary(n, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    dim, kvh = case["dim"], case["kv_heads"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "norm_rope":
        t, h = case["tokens"], case["heads"]
        rows = (_randn(g, t, h + 2 * kvh, dim) * 1.7).to(dt)       # the fused projection's rows: q | k | v
        s["q"], s["k"] = rows[:, :h], rows[:, h:h + kvh]
        s["q_weight"], s["k_weight"] = 1 + 0.2 * _randn(g, dim), 1 + 0.2 * _randn(g, dim)
        s["cos"], s["sin"] = _rotary(16384, case["rot"])
        s["positions"] = torch.randint(0, 16384, (t,), generator=g, device="cuda", dtype=torch.int32)
        return s
    new, past = _sizes(case)
    lens = [a + b for a, b in zip(new, past)]
    page, block, n = case["page"], case["block"], case["seqs"]
    per = [-(-x // page) for x in lens]
    total = sum(per)
    order = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)     # pages in no order
    table = torch.full((n, max(per)), -1, dtype=torch.int32)
    at = 0
    order = order.cpu()
    for i, p in enumerate(per):
        table[i, :p] = order[at:at + p]
        at += p
    shape = (total + 3, kvh, page, dim)
    for name in ("k", "v"):
        c = torch.empty(shape, dtype=torch.int8, device="cuda")
        for i in range(0, shape[0], 4096):
            part = c[i:i + 4096]
            part.copy_((_randn(g, *part.shape) * 33).round().clamp(-127, 127))
        s[name + "_codes"] = c
        s[name + "_scale"] = torch.exp(_randn(g, total + 3, kvh, page // block) * 0.3) * 0.03
    s["page_table"] = table.cuda()
    s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    t = cu[-1]
    s["tokens"], s["max_new"], s["max_len"] = t, max(new), max(lens)
    s["cu_tokens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "read":
        return s
    h = case["heads"]
    if case["op"] == "attention":
        s["q"] = (_randn(g, t, h, dim) * 1.3).to(dt)
        return s
    rows = (_randn(g, t, h + 2 * kvh, dim) * 1.2).to(dt)
    s["q"], s["k_new"], s["v_new"] = rows[:, :h], rows[:, h:h + kvh], rows[:, h + kvh:]
    s["q_weight"] = 1 + 0.2 * _randn(g, dim) if case["norm"] else None
    s["k_weight"] = 1 + 0.2 * _randn(g, dim) if case["norm"] else None
    s["cos"], s["sin"] = _rotary(max(lens), case["rot"])
    # what the append changed: every block that it wrote to, from its first token on
    back = [0]
    for a, b in zip(new, past):
        back.append(back[-1] + a + b % block)
    s["back"], s["back_tokens"] = torch.tensor(back, dtype=torch.int32, device="cuda"), back[-1]
    return s


# ------------------------------------------------------------------------------------------------ plain forms
EPS = 1e-6


def _plain_norm_rope(x, weight, cos, sin, interleaved):
    """x [T, H, D] in f32; cos, sin [T, rot/2]."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, x[..., 2 * half:]), -1)


def _token_places(cu, lens, total):
    """Sequence and cache position of each of `total` packed tokens that end each sequence."""
    n = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=cu.device), n, output_size=total)
    pos = (lens - n)[seq] + torch.arange(total, device=cu.device) - cu[:-1][seq]
    return seq, pos


def _plain_append(codes, scale, x, s, case):
    """x f32 [T, Hkv, D] into codes / scale, in place."""
    page, block = case["page"], case["block"]
    blocks = page // block
    seq, pos = s["places"]
    table = s["page_table"]
    pg = table[seq, pos // page].long()
    gb = pg * blocks + (pos % page) // block                         # block of each token, over all pages
    flat = scale.permute(0, 2, 1).reshape(-1, scale.shape[1])       # [page block, Hkv]
    heads = gb[:, None].expand(-1, flat.shape[1])
    amax = torch.zeros_like(flat).scatter_reduce_(0, heads, x.abs().amax(-1), "amax")
    fresh = torch.zeros_like(flat[:, 0]).scatter_reduce_(0, gb, (pos % block == 0).float(), "amax")
    old = torch.where(fresh[:, None] > 0, torch.zeros_like(flat), flat)
    need = amax / 127.0
    need = torch.where(need < TINY, torch.zeros_like(need), need)
    new = torch.maximum(old, need)
    # the codes already in each sequence's first block, rescaled where the scale grew
    cu = s["cu_tokens"].long()
    first = cu[:-1]
    p0 = pos[first]
    slot = torch.arange(block, device=x.device)
    t0 = (p0 // block * block)[:, None] + slot                       # [seqs, block] positions
    held = slot[None] < (p0 % block)[:, None]
    g0 = gb[first]
    ratio = old[g0] / torch.where(new[g0] > 0, new[g0], torch.ones_like(new[g0]))
    where = pg[first][:, None].expand_as(t0), t0 % page
    c = codes[where[0], :, where[1]].float()                         # [seqs, block, Hkv, D]
    c = torch.where(held[..., None, None], torch.round(c * ratio[:, None, :, None]), c)
    codes[where[0], :, where[1]] = c.to(torch.int8)
    d = new[gb][..., None]
    q = torch.where(d > 0, torch.round(x / torch.where(d > 0, d, torch.ones_like(d))), torch.zeros_like(x))
    codes[pg, :, pos % page] = q.clamp(-127, 127).to(torch.int8)
    scale[pg, :, pos % page // block] = new[gb]


def _plain_read(codes, scale, table, seq, pos, page, block, dt):
    pg = table[seq, pos // page].long()
    c = codes[pg, :, pos % page].float()
    return (c * scale[pg, :, pos % page // block][..., None]).to(dt)


def _plain_attention(s, case):
    page, block, kvh, dim = case["page"], case["block"], case["kv_heads"], case["dim"]
    n, group = case["seqs"], case["heads"] // case["kv_heads"]
    q, lens, cu = s["q"], s["kv_lens"].long(), s["cu_tokens"].long()
    total, mq, mk = s["tokens"], s["max_new"], s["max_len"]
    seq, pos = _token_places(cu, lens, total)
    idx = torch.arange(total, device=q.device) - cu[:-1][seq]
    padded = torch.zeros(n, mq, kvh, group, dim, device=q.device)
    padded[seq, idx] = q.float().view(total, kvh, group, dim)
    rows = padded.permute(0, 2, 1, 3, 4).reshape(n, kvh, mq * group, dim)
    pages = -(-mk // page)
    pg = s["page_table"][:, :pages].clamp(min=0).long()
    at = torch.arange(pages * page, device=q.device)
    seen = at[None] < lens[:, None]                                  # [n, L]
    kv = []
    for name in ("k", "v"):
        c = s[name + "_codes"][pg].float()                           # [n, pages, Hkv, page, D]
        c = c * s[name + "_scale"][pg].repeat_interleave(block, -1)[..., None]
        c = c.permute(0, 2, 1, 3, 4).reshape(n, kvh, pages * page, dim)
        kv.append(torch.where(seen[:, None, :, None], c, torch.zeros_like(c)))
    scores = rows @ kv[0].transpose(-1, -2) * (dim ** -0.5)
    place = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(mq, device=q.device)       # [n, mq]
    see = seen[:, None].expand(n, mq, pages * page)
    if case["causal"]:
        see = see & (at <= place[..., None])
        if case["window"]:
            see = see & (at > place[..., None] - case["window"])
    see = see.repeat_interleave(group, 1)[:, None]
    scores = scores.masked_fill(~see, -math.inf)
    top = scores.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - base)
    del scores
    z = p.sum(-1, keepdim=True)
    o = (p @ kv[1]) / torch.where(z > 0, z, torch.ones_like(z))
    lse = torch.log(z) + base
    o = o.view(n, kvh, mq, group, dim).permute(0, 2, 1, 3, 4)[seq, idx].reshape(total, kvh * group, dim)
    lse = lse.view(n, kvh, mq, group).permute(0, 2, 1, 3)[seq, idx].reshape(total, kvh * group)
    return o.to(q.dtype), lse


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm_rope":
        cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
        return [_plain_norm_rope(x.float(), w, cos, sin, case["interleaved"]).to(x.dtype)
                for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"]))]
    lens, page, block = s["kv_lens"].long(), case["page"], case["block"]
    if case["op"] == "append":
        seq, pos = _token_places(s["cu_tokens"].long(), lens, s["tokens"])
        cos, sin = s["cos"][pos], s["sin"][pos]
        q = _plain_norm_rope(s["q"].float(), s["q_weight"], cos, sin, case["interleaved"]).to(torch.bfloat16)
        k = _plain_norm_rope(s["k_new"].float(), s["k_weight"], cos, sin, case["interleaved"])
        t = dict(s, places=(seq, pos))
        _plain_append(s["k_codes"], s["k_scale"], k, t, case)
        _plain_append(s["v_codes"], s["v_scale"], s["v_new"].float(), t, case)
        seq, pos = _token_places(s["back"].long(), lens, s["back_tokens"])
        return [q] + [_plain_read(s[x + "_codes"], s[x + "_scale"], s["page_table"], seq, pos, page, block,
                                  torch.bfloat16) for x in ("k", "v")]
    if case["op"] == "read":
        seq, pos = _token_places(s["cu_tokens"].long(), lens, s["tokens"])
        return [_plain_read(s[x + "_codes"], s[x + "_scale"], s["page_table"], seq, pos, page, block,
                            DTYPES[case["dtype"]]) for x in ("k", "v")]
    return _plain_attention(s, case)


# ------------------------------------------------------------------------------------------------ one pass
def _run_own(s):
    from block_quantized_int8_q8_gb300 import api

    case = s["case"]
    if case["op"] == "norm_rope":
        return api.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos"], s["sin"], q_weight=s["q_weight"],
                                k_weight=s["k_weight"], eps=EPS, interleaved=case["interleaved"])
    cache = api.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    table, lens = s["page_table"], s["kv_lens"]
    if case["op"] == "append":
        q = api.kv_append(cache, s["k_new"], s["v_new"], table, lens, cu_tokens=s["cu_tokens"], cos=s["cos"],
                          sin=s["sin"], interleaved=case["interleaved"], k_weight=s["k_weight"], eps=EPS, q=s["q"],
                          q_weight=s["q_weight"], q_dtype=torch.bfloat16)
        k, v = api.kv_read(cache, table, lens, s["back_tokens"], cu_tokens=s["back"], dtype=torch.bfloat16)
        return [q, k, v]
    if case["op"] == "read":
        return api.kv_read(cache, table, lens, s["tokens"], cu_tokens=s["cu_tokens"], dtype=DTYPES[case["dtype"]])
    return api.attention(s["q"], cache, table, lens, max_kv_len=s["max_len"], cu_tokens=s["cu_tokens"],
                         max_tokens=s["max_new"], causal=case["causal"], window=case["window"], return_lse=True)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    dim, kvh = case["dim"], case["kv_heads"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm_rope":
        n = case["tokens"] * (case["heads"] + kvh) * dim
        return {"bytes": 2 * size * n + case["tokens"] * (4 + 4 * case["rot"]) + 8 * dim, "flops": 7 * n}
    new, past = _sizes(case)
    block, t = case["block"], sum(new)
    scale = 4.0 / block / dim                                        # bytes of scale for each code
    if case["op"] == "read":
        n = 2 * t * kvh * dim
        return {"bytes": n * (1 + scale) + n * size, "flops": n}
    if case["op"] == "append":
        n, nq = 2 * t * kvh * dim, t * case["heads"] * dim
        back = 2 * sum(a + b % block for a, b in zip(new, past)) * kvh * dim
        return {"bytes": n * size + n * (1 + scale) + nq * (size + 2) + t * 4 * case["rot"] + back * (3 + scale),
                "flops": 6 * n + 7 * nq + back}
    keys = pairs = 0
    for a, b in zip(new, past):
        if not case["causal"]:
            keys, pairs = keys + a + b, pairs + a * (a + b)
        elif not case["window"]:
            keys, pairs = keys + a + b, pairs + a * b + a * (a + 1) // 2
        else:
            w = case["window"]
            keys += min(a + b, w + a - 1)
            pairs += sum(min(w, b + i + 1) for i in range(a))
    q = t * case["heads"] * dim
    return {"bytes": 2 * keys * kvh * dim * (1 + scale) + 2 * q * size + 4 * t * case["heads"],
            "flops": 4.0 * pairs * case["heads"] * dim}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_rotate(x, weight, angles_cos, angles_sin, interleaved):
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS) * weight.double()
    out = y.clone()
    half = angles_cos.shape[-1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, d = angles_cos[:, i, None].double(), angles_sin[:, i, None].double()
        out[..., a] = y[..., a] * c - y[..., b] * d
        out[..., b] = y[..., b] * c + y[..., a] * d
    return out


def _exact_blocks(codes, scale, row, start, x, page, block):
    """The values of one sequence's blocks from the one that position `start` lies in, after x is appended."""
    out, end, at = [], start + x.shape[0], start // block * block
    while at < end:
        pg, off = int(row[at // page]), at % page
        held = max(0, start - at)
        old = scale[pg, :, off // block].double() if held else torch.zeros(x.shape[1], dtype=torch.float64,
                                                                            device=x.device)
        part = x[max(at, start) - start:min(at + block, end) - start]
        need = part.abs().amax((0, 2)) / 127.0
        new = torch.maximum(old, torch.where(need < TINY, torch.zeros_like(need), need))
        safe = torch.where(new > 0, new, torch.ones_like(new))[None, :, None]
        was = codes[pg, :, off:off + held].double().transpose(0, 1)
        both = torch.cat((torch.round(was * old[None, :, None] / safe), torch.round(part / safe)))
        out.append(both.clamp(-127, 127) * new[None, :, None])
        at += block
    return torch.cat(out)


def _exact_attention(s, case):
    page, block, kvh, dim = case["page"], case["block"], case["kv_heads"], case["dim"]
    group, table, q = case["heads"] // case["kv_heads"], s["page_table"].tolist(), s["q"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    cu = s["cu_tokens"].tolist()
    for i, length in enumerate(s["kv_lens"].tolist()):
        a, b = cu[i], cu[i + 1]
        ids = torch.tensor(table[i][:-(-length // page)], device=q.device)
        i_at = torch.arange(length - (b - a), length, device=q.device)[:, None]
        j_at = torch.arange(length, device=q.device)[None]
        hidden = torch.zeros(b - a, length, dtype=torch.bool, device=q.device)
        if case["causal"]:
            hidden = j_at > i_at
            if case["window"]:
                hidden = hidden | (j_at <= i_at - case["window"])
        for h in range(kvh):
            k, v = ((s[x + "_codes"][ids, h].double() *
                     s[x + "_scale"][ids, h].double().repeat_interleave(block, 1)[..., None]).reshape(-1, dim)[:length]
                    for x in ("k", "v"))
            for j in range(h * group, (h + 1) * group):
                e = (q[a:b, j].double() @ k.t() / math.sqrt(dim)).masked_fill(hidden, -math.inf)
                lse[a:b, j] = torch.logsumexp(e, -1)
                out[a:b, j] = torch.softmax(e, -1) @ v
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        at = s["positions"].long()
        return [_exact_rotate(s[x], s[x + "_weight"], s["cos"][at], s["sin"][at], case["interleaved"])
                for x in ("q", "k")]
    if case["op"] == "attention":
        return _exact_attention(s, case)
    page, block = case["page"], case["block"]
    lens, table = s["kv_lens"].tolist(), s["page_table"].tolist()
    cu = s["cu_tokens"].tolist()
    if case["op"] == "read":
        got = {"k": [], "v": []}
        for i, length in enumerate(lens):
            pos = torch.arange(length - (cu[i + 1] - cu[i]), length, device="cuda")
            pg = torch.tensor(table[i], device="cuda")[pos // page]
            for x in got:
                part = s[x + "_codes"][pg, :, pos % page].double()
                got[x].append(part * s[x + "_scale"][pg, :, pos % page // block].double()[..., None])
        return [torch.cat(got["k"]), torch.cat(got["v"])]
    places = torch.cat([torch.arange(n - (cu[i + 1] - cu[i]), n) for i, n in enumerate(lens)]).cuda()
    c, d = s["cos"][places], s["sin"][places]
    q = _exact_rotate(s["q"], s["q_weight"], c, d, case["interleaved"])
    k = _exact_rotate(s["k_new"], s["k_weight"], c, d, case["interleaved"])
    got = [q]
    for name, x in (("k", k), ("v", s["v_new"].double())):
        got.append(torch.cat([_exact_blocks(s[name + "_codes"], s[name + "_scale"], table[i], n - (cu[i + 1] - cu[i]),
                                            x[cu[i]:cu[i + 1]], page, block) for i, n in enumerate(lens)]))
    return got
