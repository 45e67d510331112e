"""The quantizer and the products on another stream: what they allocate belongs to that stream."""
import pytest
import torch

from block_quantized_int8_q8_gb300 import api, synth

gpu = pytest.mark.gpu


def busy(stream):
    """Keep the stream from what is queued next for some 10 ms."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


@gpu
def test_moe_workspace_and_outputs_belong_to_the_stream():
    """A busy side stream; the current one takes and fills memory of the same sizes right after each call."""
    p = synth.make_problem(synth.IQ1_M, M=24, N=128, K=256, seed=8, experts=6, slots=3)
    x, ids = torch.from_numpy(p.x).cuda(), torch.from_numpy(p.ids).cuda()
    W = torch.from_numpy(p.W.reshape(-1)).cuda()
    need = api.gemm_id_workspace_bytes(p.M, p.K, 3, p.experts)

    def step(st):
        xq = api.quantize_q8_1(x, stream=st)
        return xq, api.gemm_id(synth.IQ1_M, W, p.experts, xq, ids, p.M, p.N, p.K, stream=st)

    def fill():
        return [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
                for n in (need, api.q8_1_bytes(p.M, p.K), p.M * 3 * p.N * 4) for _ in range(3)]

    wxq, want = step(None)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(st)                                                  # both streams have memory of these sizes
    junk = fill()
    torch.cuda.synchronize()
    del junk
    busy(st)
    xq, out = step(st)
    junk = fill()
    assert not st.query()                                     # the calls have not run yet
    torch.cuda.synchronize()
    assert all((j == 0x7F).all() for j in junk)
    for views in (api.q8_1_views, api.q8_1_shadow_views):
        for a, b in zip(views(xq, p.M, p.K), views(wxq, p.M, p.K)):
            assert torch.equal(a, b)
    assert (out - want).abs().max() <= 2.0 ** -20 * want.abs().max()      # f32 sums, in any order
    assert api.read_device_errors() == 0


@gpu
def test_selftest_on_another_stream():
    st = torch.cuda.Stream()
    busy(st)
    assert api.selftest_bounded_wait(stream=st) == [0, 1, 0, 1]
    api.read_device_errors()
