"""Host-side checks of the attention operators' boundary (no GPU needed): refusals and sizes.  Arguments are refused
before any CUDA call, so the pointers here are fake and never dereferenced."""
import struct

import pytest

from block_quantized_int8_q8_gb300 import _build, api

# the structures of include/mmq.h as packed bytes (ctypes passes bytes by address)
HEADS = struct.Struct("@Pi4xqq")                              # data, dtype, token_stride, head_stride
ROTARY = struct.Struct("@PPqii")                              # cos, sin, positions, rot_dim, interleaved
CACHE = struct.Struct("@PPPPqiiii")                           # k, v, k_scale, v_scale, pages, kv_heads, head_dim, page_size, block
SEQS = struct.Struct("@PqPPi4x")                              # page_table, table_stride, kv_lens, cu_tokens, seqs
FAKE = 1 << 20
INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 6
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return api.load()


def heads(data=FAKE, dtype=BF16, ts=1024, hs=128):
    return HEADS.pack(data or 0, dtype, ts, hs)


def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=10, h=2, d=128, page=64, block=16):
    return CACHE.pack(k or 0, v or 0, ks or 0, vs or 0, pages, h, d, page, block)


def seqs(table=FAKE, stride=4, lens=FAKE, cu=FAKE, n=3):
    return SEQS.pack(table or 0, stride, lens or 0, cu or 0, n)


def rotary(cos=FAKE, sin=FAKE, positions=100, rot=128, inter=0):
    return ROTARY.pack(cos or 0, sin or 0, positions, rot, inter)


def ref(x):
    return x                                                  # packed structures go by address


def norm_rope(lib, q=heads(), hq=4, qo=heads(), k=heads(), hk=2, ko=heads(), tokens=5, dim=128, pos=FAKE,
              rot=rotary(), wq=FAKE, wk=FAKE):
    return lib.mmq_qk_norm_rope(ref(q), hq, wq, ref(qo), ref(k), hk, wk, ref(ko), tokens, dim, pos, ref(rot), 1e-6,
                                None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None, qo=None, k=None, ko=None), INVALID),
    (dict(q=None), INVALID),                                  # an output without its input
    (dict(ko=None), INVALID),
    (dict(hq=0), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(pos=None), INVALID),
    (dict(q=heads(data=None)), INVALID),
    (dict(q=heads(dtype=5)), INVALID),
    (dict(q=heads(ts=-8)), INVALID),
    (dict(dim=96), SHAPE),
    (dict(rot=rotary(rot=130)), SHAPE),
    (dict(rot=rotary(rot=136)), SHAPE),
    (dict(rot=rotary(rot=4)), SHAPE),
    (dict(rot=rotary(positions=0)), SHAPE),
    (dict(rot=rotary(cos=None)), INVALID),
    (dict(rot=rotary(sin=FAKE + 4)), ALIGN),
    (dict(q=heads(data=FAKE + 8)), ALIGN),
    (dict(q=heads(ts=1028)), ALIGN),                          # rows not 16 bytes apart
    (dict(q=heads(dtype=F32, hs=130)), ALIGN),
    (dict(pos=FAKE + 4), ALIGN),
    (dict(wq=FAKE + 4), ALIGN),
    (dict(q=heads(dtype=F16)), UNSUPPORTED),                  # q and k of two types
    (dict(qo=heads(dtype=F32)), UNSUPPORTED),
    (dict(tokens=0, pos=None), 0),
])
def test_norm_rope_refusals(lib, kw, status):
    assert norm_rope(lib, **kw) == status


def append(lib, c=cache(), s=seqs(), tokens=5, k=heads(), v=heads(), wk=None, q=None, hq=0, wq=None, qo=None, rot=None):
    return lib.mmq_kv_append(ref(c), ref(s), tokens, ref(k), ref(v), wk, ref(q), hq, wq, ref(qo), ref(rot), 1e-6, None)


CACHE_AND_SEQS = [
    (dict(c=None), INVALID),
    (dict(c=cache(d=80)), SHAPE),
    (dict(c=cache(h=0)), SHAPE),
    (dict(c=cache(pages=0)), SHAPE),
    (dict(c=cache(block=8)), SHAPE),
    (dict(c=cache(block=48, page=96)), SHAPE),
    (dict(c=cache(page=40)), SHAPE),
    (dict(c=cache(page=65536)), SHAPE),
    (dict(c=cache(pages=1 << 30, h=4)), SHAPE),
    (dict(c=cache(v=None)), INVALID),
    (dict(c=cache(ks=FAKE + 4)), ALIGN),
    (dict(s=None), INVALID),
    (dict(s=seqs(n=-1)), INVALID),
    (dict(s=seqs(n=0)), INVALID),                             # tokens of no sequence
    (dict(s=seqs(cu=None)), INVALID),                         # five tokens, three sequences
    (dict(s=seqs(table=None)), INVALID),
    (dict(s=seqs(stride=0)), SHAPE),
    (dict(s=seqs(lens=FAKE + 4)), ALIGN),
    (dict(tokens=-1), INVALID),
    (dict(tokens=1 << 31), SHAPE),
    (dict(tokens=0), 0),
    (dict(tokens=0, s=seqs(n=0)), 0),
]


@pytest.mark.parametrize("kw,status", CACHE_AND_SEQS + [
    (dict(k=None), INVALID),
    (dict(v=heads(data=FAKE + 2)), ALIGN),
    (dict(v=heads(dtype=F32)), UNSUPPORTED),
    (dict(q=heads(), qo=None, hq=4), INVALID),
    (dict(q=heads(), qo=heads(), hq=0), INVALID),
    (dict(q=heads(dtype=F16), qo=heads(), hq=4), UNSUPPORTED),
    (dict(rot=rotary(rot=256)), SHAPE),
    (dict(wk=FAKE + 8), ALIGN),
])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", CACHE_AND_SEQS + [
    (dict(k=None, v=None), INVALID),
    (dict(k=heads(dtype=F32)), UNSUPPORTED),
    (dict(k=heads(data=FAKE + 4), v=None), ALIGN),
])
def test_read_refusals(lib, kw, status):
    a = dict(c=cache(), s=seqs(), tokens=5, k=heads(), v=heads())
    a.update(kw)
    assert lib.mmq_kv_read(ref(a["c"]), ref(a["s"]), a["tokens"], ref(a["k"]), ref(a["v"]), None) == status


@pytest.mark.parametrize("kw,status", CACHE_AND_SEQS + [
    (dict(hq=0), INVALID),
    (dict(hq=7), SHAPE),                                      # not a multiple of the cache's heads
    (dict(tokens=1 << 30), SHAPE),                            # tokens * heads beyond int32
    (dict(max_tokens=0), INVALID),
    (dict(max_tokens=-1), INVALID),
    (dict(max_kv=-1), INVALID),
    (dict(max_kv=1 << 31), SHAPE),
    (dict(window=-1), INVALID),
    (dict(window=8, causal=0), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(q=heads(dtype=F32)), UNSUPPORTED),
    (dict(q=heads(data=None)), INVALID),
    (dict(out=None), INVALID),
    (dict(out=heads(ts=4)), ALIGN),
    (dict(lse=FAKE + 4), ALIGN),
    (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=-1), WORKSPACE),                           # one byte short
    (dict(ws=FAKE + 8), ALIGN),
])
def test_attention_refusals(lib, kw, status):
    a = dict(c=cache(), s=seqs(), tokens=5, hq=4, q=heads(), out=heads(), max_tokens=2, max_kv=100000, scale=0.1,
             causal=1, window=0, lse=None, ws=FAKE, ws_bytes=0)
    a.update(kw)
    need = lib.mmq_attention_workspace_bytes(5, 4, 2, 128, 3, 2, 100000)
    assert need > 0
    assert lib.mmq_attention(ref(a["q"]), a["hq"], ref(a["c"]), ref(a["s"]), a["tokens"], a["max_tokens"],
                             a["max_kv"], a["scale"], a["causal"], a["window"], ref(a["out"]), a["lse"], a["ws"],
                             need + a["ws_bytes"], None) == status


def test_workspace_sizes(lib):
    size = lib.mmq_attention_workspace_bytes
    assert size(1, 32, 8, 128, 1, 1, 100) == 0                # a short cache is not split
    assert size(1, 32, 8, 128, 1, 1, 100000) >= 32 * 128 * 4
    assert size(0, 32, 8, 128, 1, 1, 100000) == 0
    assert size(1, 32, 7, 128, 1, 1, 100000) == 0
    assert size(1, 32, 8, 96, 1, 1, 100000) == 0
    assert size(1, 32, 8, 128, 0, 1, 100000) == 0


def test_binding_refuses_what_it_cannot_pass(lib):
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 3, 64), torch.zeros(64)
    codes, scale = torch.zeros(4, 2, 32, 64, dtype=torch.int8), torch.zeros(4, 2, 2)
    for call in (lambda: api.qk_norm_rope(None, None), lambda: api.qk_norm_rope(x, None), lambda: api.qk_norm_rope(x, None, w),
                 lambda: api.KVCache(codes, codes, scale, scale), lambda: api.KVCache(codes, codes, scale, scale[:2]),
                 lambda: api.KVCache(codes.float(), codes, scale, scale), lambda: api.KVCache(1, 2, 3, 4)):
        with pytest.raises(api.MMQError):
            call()
    with pytest.raises(api.MMQError):                          # an output of another shape
        api.qk_norm_rope(x, None, q_out=x[:1])


def test_missing_binding_raises(monkeypatch, tmp_path):
    monkeypatch.setattr(api, "_bind", None)
    monkeypatch.setattr(_build, "BIND_LIB", str(tmp_path / "none.so"))
    with pytest.raises(api.MMQError):
        api._binding()
