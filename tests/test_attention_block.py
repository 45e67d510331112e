"""The attention operators as a serving loop runs them: quantized projections, append, attention, prompts and steps."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads,head_dim", [(8, 2, 128), (8, 8, 64), (4, 1, 256)])
def test_attention_block(heads, kv_heads, head_dim):
    import attention_block

    # probabilities as fp16: 2^-11 of the largest value each; bf16 queries enter both sides alike
    assert attention_block.main(heads * head_dim, heads, kv_heads, head_dim, prompts=(150, 3, 70), steps=3,
                                verbose=False) <= 2.0 ** -9
