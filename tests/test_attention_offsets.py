"""Token offsets that do not run from 0 to the number of tokens are flagged by every operator that takes them."""
import pytest
import torch

from test_attention_ops import make_cache

from block_quantized_int8_q8_gb300 import api

gpu = pytest.mark.gpu


def calls(seqs, tokens, most):
    """Each operator on `seqs` sequences of up to 64 cached tokens: name -> call with offsets."""
    g = torch.Generator().manual_seed(seqs)
    cache, table = make_cache(g, [64] * seqs, 1, 64, 64, 16)
    tb, kv = table.cuda(), torch.full((seqs,), 64, dtype=torch.int32, device="cuda")
    x = torch.randn(tokens, 1, 64, generator=g).cuda()
    q = x.bfloat16().repeat(1, 4, 1)
    return {
        "append": lambda cu: api.kv_append(cache, x, x, tb, kv, cu),
        "append with queries": lambda cu: api.kv_append(cache, x, x, tb, kv, cu, q=x),
        "read": lambda cu: api.kv_read(cache, tb, kv, tokens, cu),
        "few rows": lambda cu: api.attention(q[:, :1], cache, tb, kv, 64, cu, min(most, 16)),
        "prompts": lambda cu: api.attention(q, cache, tb, kv, 64, cu, max(most, 17)),
        "prompts, packed": lambda cu: api.attention(q, cache, tb, kv, 64, cu, 256 * 8),
    }


# more sequences than the threads of any block that looks for one, too
@gpu
@pytest.mark.parametrize("seqs", [1, 5, 129, 700])
def test_offsets_are_looked_over(seqs):
    each = 3
    tokens = seqs * each
    right = torch.arange(0, tokens + 1, each, dtype=torch.int32)
    wrong = {"starts late": (0, 1), "starts below": (0, -2), "ends early": (seqs, tokens - 1), "ends late": (seqs, tokens + 5)}
    if seqs > 1:
        wrong["falls"] = (seqs - 1, right[seqs - 2].item() - 1)
        wrong["rises over the end"] = (seqs // 2, tokens + 1)
    api.read_device_errors()
    for name, call in calls(seqs, tokens, each + 7).items():
        call(right.cuda())
        assert api.read_device_errors() == 0, name
        for what, (at, value) in wrong.items():
            cu = right.clone()
            cu[at] = value
            call(cu.cuda())
            assert api.read_device_errors() == api.DEVERR_LENGTH, (name, what)
