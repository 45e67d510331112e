"""Cases and plain forms of the operators that check a tree of drafted tokens against the 8-bit paged key/value cache.

A draft model proposes, for each sequence of a batch, a tree of continuations; the target model scores all of its tokens
in one pass and keeps one path of it.  The new tokens of a sequence are packed rows; each names the row that it
continues (`parents`: a row before it in its sequence, -1 for the cached text).  Four operators of that pass:

  tree        from parents: each token's depth, and a bit for every row that it sees (itself and its ancestors)
  append      norm and rotation of new keys and queries at the position of their depth, keys and values quantized into
              the cache in row order
  attention   softmax(q k^T) v over the cached text and, of the new tokens, those that a row sees
  keep        the rows of the accepted path moved up behind the cached text, block scales joined

The cache holds int8 codes [pages, kv heads, page size, head dim] and one f32 scale for each block of `block` tokens and
head: value = scale * code.  An append into a partly filled block keeps the block's scale unless a new value needs a
larger one; then the codes that are already there are rescaled to it.  A block whose first token is appended starts
afresh.  A block that keep moves tokens into gets the largest of the scales that its tokens had, and a code c of a
token with scale s becomes round-half-even(c * (s / that)).
"""
import math

import torch

own = False

#: a block scale below this is stored as zero (all codes zero)
TINY = 2.0 ** -63
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one chat's tree, before the first layer: latency
        {"name": "tree_1x26", "op": "tree", "seqs": 1, "new": 26, "chain": 0.2, "ragged": False},
        # a full serving batch with large trees
        {"name": "tree_256x64", "op": "tree", "seqs": 256, "new": 64, "chain": 0.3, "ragged": True},
        # one request's drafted tokens, straight from the f32 output of the quantized projection
        {"name": "append_1x32", "op": "append", "seqs": 1, "new": 32, "past": 701, "chain": 0.2, "ragged": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "norm": True, "page": 64,
         "block": 16, "dtype": "f32"},
        # a batch with a large tree each, partial rotation in adjacent pairs, no norm
        {"name": "append_64x64", "op": "append", "seqs": 64, "new": 64, "past": 900, "chain": 0.3, "ragged": True,
         "heads": 32, "kv_heads": 8, "dim": 128, "rot": 64, "interleaved": True, "norm": False, "page": 32,
         "block": 32, "dtype": "bf16"},
        # one request's accepted path: latency
        {"name": "keep_1x26", "op": "keep", "seqs": 1, "new": 26, "past": 701, "kept": 5, "chain": 0.2, "ragged": False,
         "kv_heads": 8, "dim": 128, "page": 64, "block": 16, "dtype": "bf16"},
        # a batch's accepted paths, long ones
        {"name": "keep_64x64", "op": "keep", "seqs": 64, "new": 64, "past": 900, "kept": 24, "chain": 0.3, "ragged": True,
         "kv_heads": 8, "dim": 128, "page": 32, "block": 32, "dtype": "bf16"},
        # the first tokens of a chat: a short cache, nothing but latency
        {"name": "attention_1x26_after_300", "op": "attention", "seqs": 1, "new": 26, "past": 301, "chain": 0.2,
         "ragged": False, "heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "page": 16, "block": 16,
         "dtype": "bf16"},
        # small trees over long texts: bandwidth of the cache
        {"name": "attention_16x8_after_8192", "op": "attention", "seqs": 16, "new": 8, "past": 8190, "chain": 0.3,
         "ragged": False, "heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "page": 64, "block": 16,
         "dtype": "bf16"},
        # larger trees over ragged texts: as many matrix products as the cache's bytes leave time for
        {"name": "attention_24x32_after_8192", "op": "attention", "seqs": 24, "new": 32, "past": 8192, "chain": 0.3,
         "ragged": True, "heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "page": 64, "block": 16,
         "dtype": "bf16"},
        # one request with a very long document: the work split along the cache
        {"name": "attention_1x64_after_131072", "op": "attention", "seqs": 1, "new": 64, "past": 131001, "chain": 0.2,
         "ragged": False, "heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "page": 64, "block": 64,
         "dtype": "bf16"},
        # every head with a cache of its own and small heads
        {"name": "attention_16x16_mha64", "op": "attention", "seqs": 16, "new": 16, "past": 2000, "chain": 0.3,
         "ragged": True, "heads": 32, "kv_heads": 32, "dim": 64, "window": 0, "page": 32, "block": 32,
         "dtype": "f16"},
        # large heads under a sliding window
        {"name": "attention_32x12_window_256", "op": "attention", "seqs": 32, "new": 12, "past": 6000, "chain": 0.3,
         "ragged": True, "heads": 16, "kv_heads": 4, "dim": 256, "window": 4096, "page": 64, "block": 32,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "append", "append", "keep", "keep", "attention", "attention", "attention", "attention"])
    c = {"op": op, "seqs": _log(rng, 1, 64), "chain": rng.choice([0.0, 0.2, 0.5, 0.9]), "ragged": rng.random() < 0.7}
    if op == "tree":
        c["new"] = _log(rng, 1, min(1024, 16384 // c["seqs"]))
        return c
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 8, 16])
    heads = kv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    c.update({"kv_heads": kv, "dim": dim, "page": page, "block": rng.choice([b for b in (16, 32, 64) if b <= page])})
    if op != "attention":
        c["new"] = _log(rng, 1, min(512, 4096 // c["seqs"]))
        c["past"] = 0 if rng.random() < 0.1 else _log(rng, 1, 2000)
        c["dtype"] = rng.choice(["f32", "bf16", "f16"])
        if op == "keep":
            c["kept"] = _log(rng, 1, c["new"])
        if op == "append":
            c.update({"heads": heads, "rot": rng.choice([dim, dim // 2]), "interleaved": rng.random() < 0.4,
                      "norm": rng.random() < 0.5})
        return c
    # up to 2**28 score entries in all, over a cache of up to 2**20 rows
    c["new"] = _log(rng, 1, min(512, max(1, math.isqrt((1 << 28) // (c["seqs"] * heads)))))
    most = min((1 << 28) // (c["seqs"] * c["new"] * heads), (1 << 20) // (c["seqs"] * kv)) - c["new"]
    c["past"] = 0 if rng.random() < 0.05 else _log(rng, 1, max(2, min(131072, most)))
    c.update({"heads": heads, "window": 0, "dtype": rng.choice(["bf16", "bf16", "f16"])})
    if rng.random() < 0.25:
        c["window"] = _log(rng, c["new"], max(c["new"], 4096))
    return c


def _sizes(case):
    """New tokens and cached text of every sequence: odd and ragged, from the case alone."""
    new, past = [], []
    for i in range(case["seqs"]):
        f = 1.0 if not case["ragged"] or i == 0 else ((i * 2654435761) % 1000 + 1) / 1000.0
        new.append(max(1, int(case["new"] * (0.25 + 0.75 * f))))
        past.append(int(case.get("past", 0) * f))
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


def _draft(case, seed, new):
    """Parents of all sequences' tokens: row 0 continues the text, a later row the one before it (with the probability
    `chain`) or any one before it."""
    g = torch.Generator().manual_seed(int(seed) * 7 + 3)
    rows = torch.cat([torch.arange(n) for n in new])
    u = torch.rand(rows.numel(), generator=g)
    any_row = torch.minimum((torch.rand(rows.numel(), generator=g) * rows).long(), (rows - 1).clamp(min=0))
    return torch.where(rows == 0, -1, torch.where(u < case["chain"], rows - 1, any_row)).int()


def _kept(case, seed, new):
    """The rows of each sequence's accepted path, as many as the case says: the first part of them (`chain`) in place."""
    g = torch.Generator().manual_seed(int(seed) * 7 + 3)
    out = []
    for n in new:
        count = max(1, min(n, case["kept"] * n // case["new"]))
        still = max(1, int(count * case["chain"]))
        out.append(list(range(still)) + sorted((still + torch.randperm(n - still, generator=g)[:count - still]).tolist()))
    return out


def _paths(parents, new):
    """Bits of each row's ancestors and itself, as a list of Python integers for each sequence, from the definition."""
    out, at = [], 0
    for n in new:
        seen = []
        for i, p in enumerate(parents[at:at + n].tolist()):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        out.append(seen)
        at += n
    return out


def _words(paths, words):
    flat = [(m >> (32 * w)) & 0xFFFFFFFF for seen in paths for m in seen for w in range(words)]
    return torch.tensor(flat, dtype=torch.int64).to(torch.int32).view(-1, words)


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    new, past = _sizes(case)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    t, n = cu[-1], case["seqs"]
    s["tokens"], s["max_new"] = t, max(new)
    s["cu_tokens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "tree":
        s["parents"] = _draft(case, seed, new).cuda()
        return s
    if case["op"] != "keep":
        paths = _paths(_draft(case, seed, new), new)
        s["masks"] = _words(paths, -(-max(new) // 32)).cuda()
        s["depths"] = torch.tensor([m.bit_count() - 1 for seen in paths for m in seen], dtype=torch.int32, device="cuda")
    dim, kvh, page, block = case["dim"], case["kv_heads"], case["page"], case["block"]
    lens = [a + b for a, b in zip(new, past)]
    per = [-(-x // page) for x in lens]
    total = sum(per)
    order = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32).cpu()   # pages in no order
    table = torch.full((n, max(per)), -1, dtype=torch.int32)
    at = 0
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
    s["max_len"] = max(lens)
    dt = DTYPES[case["dtype"]]
    back = [0]                                  # what the call changed: every block written to, from its first token on
    if case["op"] == "keep":
        rows = _kept(case, seed, new)
        s["counts"] = torch.tensor([len(r) for r in rows], dtype=torch.int32, device="cuda")
        most = max(len(r) for r in rows)
        s["kept"] = torch.tensor([r + [-1] * (most - len(r)) for r in rows], dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.tensor([b + len(r) for b, r in zip(past, rows)], dtype=torch.int32, device="cuda")
        for b, r in zip(past, rows):
            back.append(back[-1] + len(r) + b % block)
    elif case["op"] == "append":
        for a, b in zip(new, past):
            back.append(back[-1] + a + b % block)
    s["back"], s["back_tokens"] = torch.tensor(back, dtype=torch.int32, device="cuda"), back[-1]
    if case["op"] == "attention":
        s["q"] = (_randn(g, t, case["heads"], dim) * 1.3).to(dt)
    if case["op"] == "append":
        h = case["heads"]
        rows = (_randn(g, t, h + 2 * kvh, dim) * 1.2).to(dt)         # the fused projection's rows: q | k | v
        s["q"], s["k_new"], s["v_new"] = rows[:, :h], rows[:, h:h + kvh], rows[:, h + kvh:]
        s["q_weight"] = 1 + 0.2 * _randn(g, dim) if case["norm"] else None
        s["k_weight"] = 1 + 0.2 * _randn(g, dim) if case["norm"] else None
        s["cos"], s["sin"] = _rotary(max(lens), case["rot"])
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _plain_tree(s):
    """Reachability by squaring the matrix of steps to the parent."""
    cu, n = s["cu_tokens"].long(), s["max_new"]
    seq = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=cu.device), cu[1:] - cu[:-1], output_size=s["tokens"])
    row = torch.arange(s["tokens"], device=cu.device) - cu[:-1][seq]
    reach = torch.zeros(cu.numel() - 1, n, n + 1, device=cu.device)
    reach[seq, row, s["parents"].long()] = 1                         # (-1: the last column, the text)
    reach = reach[..., :n]
    reach[seq, row, row] = 1
    for _ in range(max(n - 1, 1).bit_length()):
        reach = (reach @ reach > 0).float()
    see = torch.zeros(s["tokens"], -(-n // 32) * 32, dtype=torch.int64, device=cu.device)
    see[:, :n] = reach[seq, row].long()
    words = (see.view(s["tokens"], -1, 32) << torch.arange(32, device=cu.device)).sum(-1)
    return [(see.sum(-1) - 1).int(), words.to(torch.int32)]


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


def _plain_append(codes, scale, x, s, case, seq, pos):
    """x f32 [T, Hkv, D] into codes / scale at the positions pos, in place."""
    page, block = case["page"], case["block"]
    blocks = page // block
    pg = s["page_table"][seq, pos // page].long()
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
    first = s["cu_tokens"].long()[:-1]
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


def _plain_keep(codes, scale, s, case):
    """Every token that the written blocks end up with, from where it was to where it goes, in place."""
    page, block = case["page"], case["block"]
    cu, table = s["cu_tokens"].long(), s["page_table"]
    base = s["kv_lens"].long() - (cu[1:] - cu[:-1])
    seq, to = _token_places(s["back"].long(), s["new_lens"].long(), s["back_tokens"])
    i = to - base[seq]
    at = torch.where(i < 0, to, base[seq] + s["kept"].long()[seq, i.clamp(min=0)])
    pg0, pg1 = table[seq, at // page].long(), table[seq, to // page].long()
    was = scale[pg0, :, at % page // block]                          # [tokens, Hkv]
    c = codes[pg0, :, at % page].float()
    gb = pg1 * (page // block) + to % page // block
    top = torch.zeros(scale.shape[0] * (page // block), was.shape[1], device=was.device)
    top = top.scatter_reduce_(0, gb[:, None].expand_as(was), was, "amax")[gb]
    ratio = was / torch.where(top > 0, top, torch.ones_like(top))
    codes[pg1, :, to % page] = torch.round(c * ratio[..., None]).to(torch.int8)
    scale[pg1, :, to % page // block] = top


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
    first = lens - (cu[1:] - cu[:-1])
    kv = []
    for name in ("k", "v"):
        c = s[name + "_codes"][pg].float()                           # [n, pages, Hkv, page, D]
        c = c * s[name + "_scale"][pg].repeat_interleave(block, -1)[..., None]
        c = c.permute(0, 2, 1, 3, 4).reshape(n, kvh, pages * page, dim)
        kv.append(torch.where((at[None] < lens[:, None])[:, None, :, None], c, torch.zeros_like(c)))
    scores = rows @ kv[0].transpose(-1, -2) * (dim ** -0.5)
    # the text before the new tokens (as far as the window at the row's depth reaches), and of these the row's ancestors
    depth = torch.zeros(n, mq, dtype=torch.int64, device=q.device)
    depth[seq, idx] = s["depths"].long()
    see = (at < first[:, None, None]).expand(n, mq, pages * page)
    if case["window"]:
        see = see & (at > (first[:, None] + depth)[..., None] - case["window"])
    bits = (s["masks"].long()[..., None] >> torch.arange(32, device=q.device) & 1).flatten(1)
    tree = torch.zeros(n, mq, bits.shape[1], dtype=torch.bool, device=q.device)
    tree[seq, idx] = bits > 0
    j = at[None] - first[:, None]                                    # row that a position holds
    drafted = (j >= 0) & (j < (cu[1:] - cu[:-1])[:, None])
    j = j.clamp(0, bits.shape[1] - 1)[:, None].expand(n, mq, pages * page)
    see = see | (drafted[:, None] & torch.gather(tree, 2, j))
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
    if case["op"] == "tree":
        return _plain_tree(s)
    if case["op"] == "attention":
        return _plain_attention(s, case)
    lens, page, block = s["kv_lens"].long(), case["page"], case["block"]
    if case["op"] == "keep":
        for x in ("k", "v"):
            _plain_keep(s[x + "_codes"], s[x + "_scale"], s, case)
        seq, pos = _token_places(s["back"].long(), s["new_lens"].long(), s["back_tokens"])
        return [_plain_read(s[x + "_codes"], s[x + "_scale"], s["page_table"], seq, pos, page, block,
                            DTYPES[case["dtype"]]) for x in ("k", "v")]
    cu = s["cu_tokens"].long()
    seq, pos = _token_places(cu, lens, s["tokens"])
    place = (lens - (cu[1:] - cu[:-1]))[seq] + s["depths"].long()
    cos, sin = s["cos"][place], s["sin"][place]
    q = _plain_norm_rope(s["q"].float(), s["q_weight"], cos, sin, case["interleaved"]).to(torch.bfloat16)
    k = _plain_norm_rope(s["k_new"].float(), s["k_weight"], cos, sin, case["interleaved"])
    _plain_append(s["k_codes"], s["k_scale"], k, s, case, seq, pos)
    _plain_append(s["v_codes"], s["v_scale"], s["v_new"].float(), s, case, seq, pos)
    seq, pos = _token_places(s["back"].long(), lens, s["back_tokens"])
    return [q] + [_plain_read(s[x + "_codes"], s[x + "_scale"], s["page_table"], seq, pos, page, block,
                              torch.bfloat16) for x in ("k", "v")]


# ------------------------------------------------------------------------------------------------ one pass
def _run_own(s):
    from block_quantized_int8_q8_gb300 import api

    case = s["case"]
    if case["op"] == "tree":
        t = api.draft_tree(s["parents"], cu_tokens=s["cu_tokens"], max_tokens=s["max_new"])
        return [t.depths, t.masks]
    cache = api.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    table, lens = s["page_table"], s["kv_lens"]
    if case["op"] == "keep":
        api.kv_keep(cache, table, lens, s["tokens"], s["kept"], s["counts"], cu_tokens=s["cu_tokens"])
        return api.kv_read(cache, table, s["new_lens"], s["back_tokens"], cu_tokens=s["back"],
                           dtype=DTYPES[case["dtype"]])
    tree = api.DraftTree(s["depths"], s["masks"])
    if case["op"] == "append":
        q = api.kv_append(cache, s["k_new"], s["v_new"], table, lens, cu_tokens=s["cu_tokens"], cos=s["cos"],
                          sin=s["sin"], interleaved=case["interleaved"], k_weight=s["k_weight"], eps=EPS, q=s["q"],
                          q_weight=s["q_weight"], q_dtype=torch.bfloat16, tree=tree)
        k, v = api.kv_read(cache, table, lens, s["back_tokens"], cu_tokens=s["back"], dtype=torch.bfloat16)
        return [q, k, v]
    return api.attention(s["q"], cache, table, lens, max_kv_len=s["max_len"], cu_tokens=s["cu_tokens"],
                         max_tokens=s["max_new"], window=case["window"], return_lse=True, tree=tree)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    new, past = _sizes(case)
    t, words = sum(new), -(-max(new) // 32)
    if case["op"] == "tree":
        return {"bytes": t * (8 + 4 * words), "flops": t * words}
    dim, kvh, block = case["dim"], case["kv_heads"], case["block"]
    size = 4 if case["dtype"] == "f32" else 2
    scale = 4.0 / block / dim                                        # bytes of scale for each code
    if case["op"] == "keep":
        # the rows of the path that are not in place, read and written; the written blocks read back
        rows = _kept(case, 0, new)
        moved = sum(len(r) - max(1, int(len(r) * case["chain"])) for r in rows)
        back = sum(len(r) + b % block for r, b in zip(rows, past))
        n, m = 2 * kvh * dim * moved, 2 * kvh * dim * back
        return {"bytes": n * (2 + 2 * scale) + m * (1 + scale + size), "flops": 2 * n + m}
    if case["op"] == "append":
        n, nq = 2 * t * kvh * dim, t * case["heads"] * dim
        back = 2 * sum(a + b % block for a, b in zip(new, past)) * kvh * dim
        return {"bytes": n * size + n * (1 + scale) + nq * (size + 2) + t * 4 * (case["rot"] + 1) + back * (3 + scale),
                "flops": 6 * n + 7 * nq + back}
    keys = pairs = 0
    for a, b in zip(new, past):
        w = min(b, case["window"]) if case["window"] else b
        keys, pairs = keys + a + w, pairs + a * w + min(a * (a + 1) // 2, 8 * a)
    q = t * case["heads"] * dim
    return {"bytes": 2 * keys * kvh * dim * (1 + scale) + 2 * q * size + 4 * t * (case["heads"] + words + 1),
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


def _exact_kept(codes, scale, row, base, rows, page, block):
    """The values of one sequence's blocks from the one that position `base` lies in, with the kept rows moved up."""
    out, at = [], base // block * block
    src = list(range(at, base)) + [base + r for r in rows]
    while src:
        part, src = src[:block], src[block:]
        was = torch.stack([scale[int(row[p // page]), :, p % page // block].double() for p in part])
        c = torch.stack([codes[int(row[p // page]), :, p % page].double() for p in part])
        top = was.amax(0)
        safe = torch.where(top > 0, top, torch.ones_like(top))
        # the ratio is a rounded f32 number, as the scales are: it decides which way halves go
        ratio = (was / safe).float().double()
        out.append(torch.round(c * ratio[..., None]) * top[None, :, None])
    return torch.cat(out) if out else codes.new_zeros((0,) + codes.shape[1::2], dtype=torch.float64)


def _exact_attention(s, case):
    page, block, kvh, dim = case["page"], case["block"], case["kv_heads"], case["dim"]
    group, table, q = case["heads"] // case["kv_heads"], s["page_table"].tolist(), s["q"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    cu, words, depth = s["cu_tokens"].tolist(), s["masks"].cpu().numpy().view("uint32"), s["depths"]
    for i, length in enumerate(s["kv_lens"].tolist()):
        a, b = cu[i], cu[i + 1]
        first = length - (b - a)
        ids = torch.tensor(table[i][:-(-length // page)], device=q.device)
        hidden = torch.zeros(b - a, length, dtype=torch.bool)
        for r in range(b - a):
            hidden[r, first:] = torch.tensor([not words[a + r, j // 32] >> (j % 32) & 1 for j in range(b - a)])
        hidden = hidden.to(q.device)
        if case["window"]:
            lowest = (first + depth[a:b].long() - case["window"])[:, None]
            hidden |= (torch.arange(length, device=q.device)[None] <= lowest) & \
                (torch.arange(length, device=q.device)[None] < first)
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
    new, past = _sizes(case)
    if case["op"] == "tree":
        paths = _paths(s["parents"].cpu(), new)
        depths = torch.tensor([m.bit_count() - 1 for seen in paths for m in seen], dtype=torch.int32, device="cuda")
        return [depths, _words(paths, -(-max(new) // 32)).cuda()]
    if case["op"] == "attention":
        return _exact_attention(s, case)
    page, block = case["page"], case["block"]
    table, cu = s["page_table"].tolist(), s["cu_tokens"].tolist()
    if case["op"] == "keep":
        rows = [r[:c] for r, c in zip(s["kept"].tolist(), s["counts"].tolist())]
        return [torch.cat([_exact_kept(s[x + "_codes"], s[x + "_scale"], table[i], past[i], rows[i], page, block)
                           for i in range(case["seqs"])]) for x in ("k", "v")]
    places = torch.cat([torch.full((n,), p) for n, p in zip(new, past)]).cuda() + s["depths"].long()
    c, d = s["cos"][places], s["sin"][places]
    q = _exact_rotate(s["q"], s["q_weight"], c, d, case["interleaved"])
    k = _exact_rotate(s["k_new"], s["k_weight"], c, d, case["interleaved"])
    got = [q]
    for name, x in (("k", k), ("v", s["v_new"].double())):
        got.append(torch.cat([_exact_blocks(s[name + "_codes"], s[name + "_scale"], table[i], past[i],
                                            x[cu[i]:cu[i + 1]], page, block) for i in range(case["seqs"])]))
    return got
