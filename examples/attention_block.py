"""An attention block on quantized weights and an 8-bit cache, as a serving loop runs it.

    x -> q8_1 -> Q4_0 product (fused q | k | v) -> norm, rotation, append to the paged cache -> attention
      -> q8_1 -> Q4_0 product (output projection) -> + x

One call of `step` takes the new tokens of every sequence of a batch: whole prompts first, then one token each.  Run it
to see both, checked against plain torch arithmetic on the cache's own values:

    python examples/attention_block.py
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

from block_quantized_int8_q8_gb300 import api, synth


class AttentionBlock:
    """Weights, rotation table and paged cache of one block.  `pages` is shared by all sequences; a page table row lists
    the pages of one."""

    def __init__(self, hidden, heads, kv_heads, head_dim, pages, max_positions, page_size=64, block=16, seed=0):
        self.hidden, self.heads, self.kv_heads, self.head_dim = hidden, heads, kv_heads, head_dim
        self.width = (heads + 2 * kv_heads) * head_dim
        qkv = synth.make_problem(synth.Q4_0, M=1, N=self.width, K=hidden, seed=seed)
        out = synth.make_problem(synth.Q4_0, M=1, N=hidden, K=heads * head_dim, seed=seed + 1)
        self.w_qkv = torch.from_numpy(qkv.W.reshape(-1)).cuda()
        self.w_out = torch.from_numpy(out.W.reshape(-1)).cuda()
        self.q_norm = torch.ones(head_dim, device="cuda")
        self.k_norm = torch.ones(head_dim, device="cuda")
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda") / head_dim)
        angle = torch.arange(max_positions, device="cuda")[:, None] * inv
        self.cos, self.sin = angle.cos(), angle.sin()
        self.cache = api.KVCache.empty(pages, kv_heads, head_dim, page_size, block)

    def project(self, w, x, rows):
        return api.gemm(synth.Q4_0, w, api.quantize_q8_1(x), x.shape[0], rows, x.shape[1])

    def step(self, x, page_table, kv_lens, max_kv_len, cu_tokens=None, max_tokens=1):
        """x f32 [tokens, hidden], the batch's new tokens back to back; kv_lens: cached tokens of each sequence, these
        included.  Nothing waits for the host.  Returns the block's output and the queries and attention inside."""
        rows = self.project(self.w_qkv, x, self.width).view(-1, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        q = api.kv_append(self.cache, k, v, page_table, kv_lens, cu_tokens, self.cos, self.sin, k_weight=self.k_norm, q=q,
                          q_weight=self.q_norm, q_dtype=torch.bfloat16)
        a = api.attention(q, self.cache, page_table, kv_lens, max_kv_len, cu_tokens, max_tokens, out_dtype=torch.float32)
        return x + self.project(self.w_out, a.view(x.shape[0], -1), self.hidden), q, a


def plain_attention(block, q, page_table, kv_lens, new):
    """The same attention from the cache's values, in f32 with plain torch operations, sequence by sequence."""
    out, at, group = [], 0, block.heads // block.kv_heads
    for i, (length, n) in enumerate(zip(kv_lens.tolist(), new)):
        one, cu = kv_lens[i:i + 1].clone(), torch.tensor([0, length], dtype=torch.int32, device="cuda")
        k, v = api.kv_read(block.cache, page_table[i:i + 1].clone(), one, length, cu, torch.float32)
        k, v = (t.repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))
        s = q[at:at + n].float().transpose(0, 1) @ k.transpose(1, 2) * block.head_dim ** -0.5
        place = torch.arange(length - n, length, device="cuda")[:, None]
        s = s.masked_fill(torch.arange(length, device="cuda") > place, float("-inf"))
        out.append((torch.softmax(s, -1) @ v).transpose(0, 1))
        at += n
    return torch.cat(out)


def main(hidden=1024, heads=8, kv_heads=2, head_dim=128, prompts=(300, 45, 129), steps=4, verbose=True):
    """Prompts, then single tokens.  Returns the largest relative difference from the plain attention."""
    n, page = len(prompts), 64
    most = max(prompts) + steps
    per = -(-most // page)
    block = AttentionBlock(hidden, heads, kv_heads, head_dim, n * per, most, page)
    table = torch.randperm(n * per).view(n, per).to(torch.int32).cuda()          # pages in any order
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + list(prompts), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    worst = 0.0

    def look(name, q, a, new):
        nonlocal worst
        want = plain_attention(block, q, table, lens, new)
        far = float((a - want).abs().max() / want.abs().max())
        worst = max(worst, far)
        if verbose:
            print(f"{name}: {sum(new)} tokens, {lens.tolist()} cached, largest difference {far:.1e} of the output's scale")

    x = torch.randn(sum(prompts), hidden, device="cuda", generator=g)
    y, q, a = block.step(x, table, lens, most, cu, max(prompts))
    look("prompts", q, a, list(prompts))
    for i in range(steps):
        lens += 1
        x = y[cu[1:].long() - 1] if i == 0 else y                                # the last token's output, fed back
        y, q, a = block.step(x.contiguous(), table, lens, most)
        look(f"token {i + 1}", q, a, [1] * n)
    assert torch.isfinite(y).all() and api.read_device_errors() == 0
    return worst


if __name__ == "__main__":
    main()
