"""Attention and its cache at the edges of their arguments and inputs (tolerances as in test_attention_ops.py)."""
import sys

import pytest
import torch

from test_attention_ops import check_attention, make_cache, offsets

from block_quantized_int8_q8_gb300 import api

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("n", [[1, 1], [40, 150]])
def test_windows_that_hide_nothing(n):
    """The largest windows are none: the same bits, with caches that are cut in parts."""
    lens = [9001, 700]
    want = check_attention(lens, n, 4, 1, 128, 64, 16)
    for window in (9001, 1 << 31, sys.maxsize):
        assert torch.equal(check_attention(lens, n, 4, 1, 128, 64, 16, window=window), want)
