"""The operators on a tree of drafted tokens at the edges of what their documentation allows.  Tolerances as in
test_draft_tree.py."""
import pytest
import torch

import test_draft_tree as T
from test_attention_ops import make_cache

from block_quantized_int8_q8_gb300 import api

gpu = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ nothing to do
@gpu
def test_an_empty_batch_goes_through_every_operator():
    g = torch.Generator().manual_seed(1)
    cache, table = make_cache(g, [30, 40], 2, 64, 16, 16)
    before = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    rows = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    tb, kv, cu = table.cuda(), T.i32([30, 40]), T.i32([0, 0, 0])
    tree = api.draft_tree(T.i32([]), cu, 5)
    q = api.kv_append(cache, rows[:, 4:6], rows[:, 6:], tb, kv, cu, q=rows[:, :4], tree=tree)
    out, lse = api.attention(q, cache, tb, kv, 100, cu, 5, tree=tree, return_lse=True)
    assert q.shape == out.shape == (0, 4, 64) and lse.shape == (0, 4)
    api.kv_keep(cache, tb, kv, 0, T.i32([]).view(2, 0), T.i32([0, 0]), cu)
    assert api.read_device_errors() == 0
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


@gpu
def test_keep_of_no_rows():
    """No sequence keeps a token; a count that asks for one all the same is flagged."""
    g = torch.Generator().manual_seed(1)
    cache, table = make_cache(g, [30, 40], 2, 64, 16, 16)
    before = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    tb, kv, cu = table.cuda(), T.i32([30, 40]), T.i32([0, 6, 10])
    none = T.i32([]).view(2, 0)
    api.kv_keep(cache, tb, kv, 10, none, T.i32([0, 0]), cu)
    assert api.read_device_errors() == 0
    api.kv_keep(cache, tb, kv, 10, none, T.i32([0, 1]), cu)
    assert api.read_device_errors() == api.DEVERR_DRAFT
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))
