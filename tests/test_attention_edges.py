"""Attention and its cache at the edges of their arguments and inputs (tolerances as in test_attention_ops.py)."""
import copy
import math
import struct
import sys

import pytest
import torch

from test_attention_ops import assert_close, check_attention, make_cache, offsets, rotary_tables

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


def busy(stream):
    """Keep the stream from what is queued next for some 10 ms."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


@gpu
@pytest.mark.parametrize("n", [1, 70])
def test_workspace_stays_with_the_call_s_stream(n):
    """Neither output nor workspace given, another stream that is busy: memory taken and filled at once on the current
    stream is not the call's."""
    cache, table = make_cache(torch.Generator().manual_seed(n), [9001], 1, 128, 64, 16)
    q = torch.randn(n, 4, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    kv, cu, tb = torch.tensor([9001], dtype=torch.int32, device="cuda"), offsets([n]).cuda(), table.cuda()
    want, wlse = api.attention(q, cache, tb, kv, 9001, cu, n, return_lse=True)
    size = api.attention_workspace_bytes(n, 4, 1, 128, 1, n, 9001)
    assert size > 0
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        api.attention(q, cache, tb, kv, 9001, cu, n, stream=st)          # both streams have memory of these sizes
        junk = [torch.full((size // 4,), float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        busy(st)
        out, lse = api.attention(q, cache, tb, kv, 9001, cu, n, return_lse=True, stream=st)
        junk = [torch.full((size // 4,), float("nan"), device="cuda") for _ in range(4)]
        assert not st.query()                                 # the call has not run yet
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse) and all(j.isnan().all() for j in junk)


@gpu
def test_outputs_take_no_memory_that_another_stream_still_reads():
    g = torch.Generator().manual_seed(3)
    cache, table = make_cache(g, [64], 2, 64, 64, 16)
    tb, kv, cu = table.cuda(), torch.tensor([64], dtype=torch.int32, device="cuda"), offsets([64]).cuda()
    x = torch.randn(64, 2, 64, generator=g).cuda()
    w = torch.ones(64, device="cuda")
    q = x.bfloat16()
    calls = {
        "norm": lambda st: api.qk_norm_rope(x, None, q_weight=w, stream=st)[0],
        "append": lambda st: api.kv_append(cache, x, x, tb, kv, cu, q=x, q_weight=w, stream=st),
        "read": lambda st: api.kv_read(cache, tb, kv, 64, cu, torch.float32, stream=st)[0],
        "attention": lambda st: api.attention(q, cache, tb, kv, 64, cu, 64, out_dtype=torch.float32, stream=st),
    }
    for name, call in calls.items():
        st, mine = torch.cuda.Stream(), torch.cuda.current_stream()
        torch.cuda.synchronize()
        call(st)                                              # the stream has memory of this size
        torch.cuda.synchronize()
        held = [torch.full_like(x, float(i)) for i in range(8)]
        copies = [torch.empty_like(x) for _ in held]
        torch.cuda.synchronize()
        busy(mine)
        for h, c in zip(held, copies):
            c.copy_(h)                                        # queued behind the wait
        held = h = None                                       # given back while still to be read
        outs = [call(st) for _ in range(4)]
        st.synchronize()
        assert not mine.query(), name
        mine.synchronize()
        for i, c in enumerate(copies):
            assert (c == i).all(), name
        want = call(None)
        for o in outs:
            assert torch.equal(o, want), name


@gpu
@pytest.mark.parametrize("D,group", [(64, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("ot", [torch.bfloat16, torch.float32])
def test_prompt_rows_without_any_position_are_zeros(D, group, ot):
    """Many blocks of rows for which there is no cache tile: their outputs leave while other rows' queries still come in
    from far apart."""
    n, seqs, heads = 256 // group + 5, 64, 4
    cache = api.KVCache.empty(4, heads // group, D, 64, 16)
    wide = torch.randn(seqs * n, 64, D, device="cuda", generator=torch.Generator("cuda").manual_seed(D)).bfloat16() + 3
    q = wide[:, ::16]                                         # heads far apart in memory
    table = torch.zeros(seqs, 1, dtype=torch.int32, device="cuda")
    kv = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    cu = offsets([n] * seqs).cuda()
    for _ in range(10):
        out = torch.full((seqs * n, heads, D), 5.0, dtype=ot, device="cuda")
        _, lse = api.attention(q, cache, table, kv, 64, cu, n, out=out, return_lse=True)
        assert (out == 0).all() and torch.isneginf(lse).all()
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("where", [0, 20000, 40003])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 20])
def test_one_strong_position_over_a_long_cache_of_weak_ones(n, D, where):
    """One position 2^16 to 2^34 above 40003 others of equal score and opposite value: together these weigh 2^-1 to 2^-19
    of it, and keep that share.  Each keeps fp16's bits or is rounded to 2^-36 of the strong one, 2^-20 for all of them, so
    the tolerance stays.  There are as many sequences as leave the cache of prompts in one piece."""
    L, seqs, B = 40004, 160, 16
    pages = -(-L // 64)
    cache = api.KVCache.empty(pages, 1, D, 64, B)
    cache.k.zero_()
    cache.v.fill_(-127)
    cache.k_scale.fill_(1 / 127)
    cache.v_scale.fill_(1 / 127)
    cache.k[where // 64, 0, where % 64, 0] = 127
    cache.v[where // 64, 0, where % 64] = 127
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(seqs, pages).contiguous()
    kv = torch.full((seqs,), L, dtype=torch.int32, device="cuda")
    q = torch.zeros(seqs * n, 1, D, dtype=torch.float16)
    q[:, 0, 0] = torch.linspace(16, 34, seqs * n).half()      # powers of two: scale ln 2
    scale = math.log(2)
    out, lse = api.attention(q.cuda(), cache, table, kv, L, offsets([n] * seqs).cuda(), n, scale=scale, causal=False,
                             out_dtype=torch.float32, return_lse=True)
    unit = float(torch.tensor(1 / 127, dtype=torch.float32))
    s = q[:, 0, 0].double() * 127 * unit * float(torch.tensor(scale, dtype=torch.float32))
    w = (L - 1) * torch.exp(-s)
    want = (127 * unit * (1 - w) / (1 + w))[:, None, None].expand(-1, 1, D)
    assert_close(out, want, torch.full_like(want, 2.0 ** -11 + 2.0 ** -16))
    assert_close(lse, (s + torch.log1p(w))[:, None], (2.0 ** -18 + 2.0 ** -20 * s)[:, None])
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("base", [-8e6, -2e6, 1e6, 2e6, 4e6, 8e6])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 40])
def test_scores_of_large_magnitude(n, D, base):
    """Scores of up to 2^23 in magnitude, where f32 steps by up to a binary order: equal ones average, and ones that differ
    by up to 2^20 weigh whatever f32 leaves of their differences, within the largest value."""
    L, seqs = 1500, 64
    g = torch.Generator().manual_seed(int(abs(base)) + D)
    cache, table = make_cache(g, [L], 1, D, 64, 16)
    cache.k_scale.fill_(1 / 64)
    cache.v_scale.fill_(1 / 64)
    cache.k[..., 0] = 64
    table = table.repeat(seqs, 1).cuda()
    kv, cu = torch.full((seqs,), L, dtype=torch.int32, device="cuda"), offsets([n] * seqs).cuda()
    ref = cache.v.double().cpu()[table[0, :-(-L // 64)].long().cpu()][:, 0].reshape(-1, D)[:L] / 64
    vmax = float(ref.abs().max())
    q = torch.zeros(seqs * n, 2, D, dtype=torch.bfloat16)
    q[..., 0] = base
    out, lse = api.attention(q.cuda(), cache, table, kv, L, cu, n, scale=1.0, causal=False, out_dtype=torch.float32,
                             return_lse=True)
    want = ref.mean(0).expand(seqs * n, 2, D)
    assert_close(out, want, torch.full_like(want, vmax * (2.0 ** -11 + 2.0 ** -16)))
    s = q[..., 0].double() + math.log(L)
    assert_close(lse, s, 2.0 ** -18 + 2.0 ** -20 * s.abs())
    q[..., 1:] = torch.randn(seqs * n, 2, D - 1, generator=g) * 2
    out = api.attention(q.cuda(), cache, table, kv, L, cu, n, scale=1.0, causal=False, out_dtype=torch.float32)
    assert torch.isfinite(out).all() and float(out.abs().max()) <= vmax * (1 + 2.0 ** -10)
    assert api.read_device_errors() == 0


@gpu
def test_copies_of_a_cache():
    cache, table = make_cache(torch.Generator().manual_seed(1), [64], 1, 64, 64, 16)
    kv, cu, tb = torch.tensor([64], dtype=torch.int32, device="cuda"), offsets([64]).cuda(), table.cuda()
    shallow, deep = copy.copy(cache), copy.deepcopy(cache)
    assert shallow.k is cache.k and deep.k.data_ptr() != cache.k.data_ptr()
    before = api.kv_read(cache, tb, kv, 64, cu)
    x = torch.full((64, 1, 64), 9.0, device="cuda")
    api.kv_append(cache, x, x, tb, kv, cu)
    for c, want in ((shallow, api.kv_read(cache, tb, kv, 64, cu)), (deep, before)):
        assert all(torch.equal(a, b) for a, b in zip(api.kv_read(c, tb, kv, 64, cu), want))


@gpu
def test_tensors_of_another_device_are_refused(monkeypatch):
    """Tensors that claim to lie on the next device (without memory) in each place of each call."""
    from torch._subclasses import fake_tensor
    from torch._subclasses.fake_tensor import FakeTensorMode

    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda device: None)      # there need not be such a device
    far = torch.cuda.current_device() + 1
    mode = FakeTensorMode()

    def there(t):
        with mode:
            return torch.empty(t.shape, dtype=t.dtype, device=f"cuda:{far}")

    cache, table = make_cache(torch.Generator().manual_seed(1), [64], 2, 64, 64, 16)
    x = torch.randn(64, 2, 64, device="cuda")
    cos, sin = (t.cuda() for t in rotary_tables(64, 64))
    w, pos = torch.ones(64, device="cuda"), torch.arange(64, dtype=torch.int32, device="cuda")
    tb, kv, cu = table.cuda(), torch.tensor([64], dtype=torch.int32, device="cuda"), offsets([64]).cuda()
    ws = torch.empty(1024, dtype=torch.uint8, device="cuda")
    calls = (
        (api.qk_norm_rope, dict(q=x, k=x, positions=pos, cos=cos, sin=sin, q_weight=w, k_weight=w, q_out=x, k_out=x)),
        (api.kv_append, dict(cache=cache, k=x, v=x, page_table=tb, kv_lens=kv, cu_tokens=cu, cos=cos, sin=sin,
                             k_weight=w, q=x, q_weight=w, q_out=x.clone())),
        (api.kv_read, dict(cache=cache, page_table=tb, kv_lens=kv, tokens=64, cu_tokens=cu)),
        (api.attention, dict(q=x.half(), cache=cache, page_table=tb, kv_lens=kv, max_kv_len=64, cu_tokens=cu,
                             max_tokens=64, out=x.clone(), workspace=ws)),
    )
    elsewhere = copy.copy(cache)
    object.__setattr__(elsewhere, "_packed", cache._packed[:-8] + struct.pack("=ii", far, 0))
    for call, given in calls:
        call(**given)
        for name, value in given.items():
            if name == "cache" or torch.is_tensor(value):
                with pytest.raises(api.MMQError, match="device"):
                    call(**{**given, name: elsewhere if name == "cache" else there(value)})
    assert api.read_device_errors() == 0


def check_long_caches(L, n, causal, D):
    """Sequences of n[i] new tokens over one cache of L tokens that they share, the largest scores early for some rows and
    late for others."""
    seqs, total, pages = len(n), sum(n), -(-L // 64)
    g = torch.Generator("cuda").manual_seed(D + seqs)
    cache = api.KVCache.empty(pages, 1, D, 64, 16)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.copy_((torch.randn(c.shape, device="cuda", generator=g) * 40).round().clamp(-127, 127))
        s.uniform_(0.001, 0.02, generator=g)
    tilt = torch.linspace(-100, 100, pages * 64, device="cuda").view(pages, 1, 64)
    cache.k[..., 0] = tilt.round().to(torch.int8)
    cache.k_scale.fill_(0.01)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(seqs, pages).contiguous()
    kv, cu = torch.full((seqs,), L, dtype=torch.int32, device="cuda"), offsets(n).cuda()
    q = torch.randn(total, 1, D, device="cuda", generator=g)
    q[:, 0, 0] = torch.linspace(-150, 150, total, device="cuda")[torch.randperm(total, device="cuda", generator=g)]
    q = q.bfloat16()
    out, lse = api.attention(q, cache, table, kv, L, cu, max(n), scale=D ** -0.5, causal=causal, out_dtype=torch.float32,
                             return_lse=True)
    one, cu1 = kv[:1].clone(), offsets([L]).cuda()
    k, v = (t[:, 0].double() for t in api.kv_read(cache, table[:1].clone(), one, L, cu1, torch.float32))
    place = torch.cat([torch.arange(L - m, L, device="cuda") for m in n])
    for a in range(0, total, 300):
        s = q[a:a + 300, 0].double() @ k.T * D ** -0.5
        if causal:
            s.masked_fill_(torch.arange(L, device="cuda") > place[a:a + 300, None], -math.inf)
        want = (torch.softmax(s, -1) @ v).cpu()
        wlse = torch.logsumexp(s, -1).cpu()
        # scores reach 2^7 here, four times those that 2^-16 is stated for
        assert_close(out[a:a + 300, 0], want, torch.full_like(want, float(v.abs().max()) * (2.0 ** -11 + 2.0 ** -14)))
        assert_close(lse[a:a + 300, 0], wlse, 2.0 ** -18 + 2.0 ** -20 * wlse.abs())
    assert api.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L,seqs,causal", [(70001, 160, False), (100003, 100, True), (70001, 40, True)])
def test_sums_put_aside_over_long_caches(L, seqs, causal, D):
    """Prompts over caches so long that sums are put aside once or twice, in one piece and in parts that are joined."""
    check_long_caches(L, [18] * seqs, causal, D)


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_sums_put_aside_in_a_mixed_batch(causal, D):
    """Rows numbered through the batch: a prompt, single tokens and empty sequences over a cache of three such sums."""
    check_long_caches(100003, [1, 0] * 60 + [700] + [1, 2, 0] * 40, causal, D)
