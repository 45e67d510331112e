"""Thin Python binding of libmmq_gb300.so (argument marshalling only).

Every function forwards device pointers, sizes and the current CUDA stream to the C ABI declared in
include/mmq.h; all arithmetic runs in the library's sm_103a kernels.  PyTorch is used only for device
memory and streams.  If the library is missing or fails to load, every call raises: there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import _build

Q8_0, Q4_0, Q4_K, IQ1_M, W8A8, Q6_K = 0, 1, 2, 3, 4, 5
DEVERR_TIMEOUT, DEVERR_EXPERT_ID, DEVERR_DUP_EXPERT = 1, 2, 4
DEVERR_PAGE, DEVERR_POSITION, DEVERR_LENGTH = 8, 16, 32

#: every symbol include/mmq.h declares
EXPORTS = ("mmq_status_string", "mmq_last_cuda_error", "mmq_q8_1_bytes", "mmq_weight_bytes", "mmq_w8a8_act_bytes", "mmq_quantize_q8_1",
           "mmq_gemm", "mmq_gemm_id_workspace_bytes", "mmq_gemm_id", "mmq_gemm_debug_partials",
           "mmq_gemm_debug_block_sums", "mmq_selftest_bounded_wait",
           "mmq_read_device_errors", "mmq_gemm_id_noalloc", "mmq_q8_1_prepare",
           "mmq_qk_norm_rope", "mmq_kv_append", "mmq_kv_read", "mmq_attention_workspace_bytes", "mmq_attention")
NOALLOC_SCRATCH_BYTES = 1 << 20

_lib = None


class MMQError(RuntimeError):
    pass


# The structures of include/mmq.h as packed bytes, which ctypes passes by address (a ctypes.Structure takes three
# times as long to fill, and these are made on every call).
_HEADS = struct.Struct("@Pi4xqq")                # mmq_heads: data, dtype, token_stride, head_stride
_ROTARY = struct.Struct("@PPqii")                # mmq_rotary: cos, sin, positions, rot_dim, interleaved
_CACHE = struct.Struct("@PPPPqiiii")             # mmq_kv_cache: k, v, k_scale, v_scale, pages, kv_heads, head_dim, page_size, block
_SEQS = struct.Struct("@PqPPi4x")                # mmq_kv_seqs: page_table, table_stride, kv_lens, cu_tokens, seqs


def library_path() -> str:
    return _build.LIB


def load():
    """Load the CUDA library (it must have been built by __graft_entry__.build() or _build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise MMQError(f"CUDA library not built: {path} is missing (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.mmq_status_string.argtypes = [I]
    lib.mmq_status_string.restype = ctypes.c_char_p
    lib.mmq_last_cuda_error.argtypes = []
    lib.mmq_last_cuda_error.restype = ctypes.c_char_p
    lib.mmq_q8_1_bytes.argtypes = [I64, I64]
    lib.mmq_q8_1_bytes.restype = SZ
    lib.mmq_weight_bytes.argtypes = [I, I64, I64]
    lib.mmq_weight_bytes.restype = SZ
    lib.mmq_w8a8_act_bytes.argtypes = [I64, I64]
    lib.mmq_w8a8_act_bytes.restype = SZ
    lib.mmq_quantize_q8_1.argtypes = [P, I64, I64, P, P]
    lib.mmq_q8_1_prepare.argtypes = [P, I64, I64, P]
    lib.mmq_q8_1_prepare.restype = I
    lib.mmq_quantize_q8_1.restype = I
    lib.mmq_gemm.argtypes = [I, P, P, P, I64, I64, I64, P]
    lib.mmq_gemm.restype = I
    lib.mmq_gemm_id_workspace_bytes.argtypes = [I64, I64, I, I]
    lib.mmq_gemm_id_workspace_bytes.restype = SZ
    lib.mmq_gemm_id.argtypes = [I, P, I, P, P, I, P, I64, I64, I64, P, SZ, P]
    lib.mmq_gemm_id.restype = I
    lib.mmq_gemm_debug_partials.argtypes = [I, P, P, P, I64, I64, I64, P]
    lib.mmq_gemm_debug_partials.restype = I
    lib.mmq_gemm_debug_block_sums.argtypes = [I, P, P, P, I64, I64, I64, P]
    lib.mmq_gemm_debug_block_sums.restype = I
    lib.mmq_selftest_bounded_wait.argtypes = [P, P]
    lib.mmq_selftest_bounded_wait.restype = I
    lib.mmq_gemm_id_noalloc.argtypes = [I, P, I, P, P, I, P, I64, I64, I64, P]
    lib.mmq_gemm_id_noalloc.restype = I
    lib.mmq_read_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint), P]
    lib.mmq_read_device_errors.restype = I
    F = ctypes.c_float
    lib.mmq_qk_norm_rope.argtypes = [P, I, P, P, P, I, P, P, I64, I, P, P, F, P]
    lib.mmq_kv_append.argtypes = [P, P, I64, P, P, P, P, I, P, P, P, F, P]
    lib.mmq_kv_read.argtypes = [P, P, I64, P, P, P]
    lib.mmq_attention_workspace_bytes.argtypes = [I64, I, I, I, I, I64, I64]
    lib.mmq_attention_workspace_bytes.restype = SZ
    lib.mmq_attention.argtypes = [P, I, P, P, I64, I64, I64, F, I, I64, P, P, P, SZ, P]
    for f in (lib.mmq_qk_norm_rope, lib.mmq_kv_append, lib.mmq_kv_read, lib.mmq_attention):
        f.restype = I
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = load().mmq_status_string(rc).decode()
        if rc == 5:
            msg += "; " + load().mmq_last_cuda_error().decode()
        raise MMQError(f"{what}: status {rc} ({msg})")


def _stream(stream) -> int:
    # the current stream's handle straight from the runtime: building torch's stream object for it takes 2.8 us
    return stream.cuda_stream if stream is not None else _raw_stream(_current_device())


_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise MMQError("expected a contiguous CUDA tensor")
    return t.data_ptr()


# ------------------------------------------------------------------------------------------ sizes / layouts
def q8_1_bytes(M: int, K: int) -> int:
    return int(load().mmq_q8_1_bytes(M, K))


def weight_bytes(wtype: int, N: int, K: int) -> int:
    return int(load().mmq_weight_bytes(wtype, N, K))


def w8a8_act_bytes(M: int, K: int) -> int:
    return int(load().mmq_w8a8_act_bytes(M, K))


def gemm_id_workspace_bytes(M: int, K: int, slots: int, experts: int) -> int:
    return int(load().mmq_gemm_id_workspace_bytes(M, K, slots, experts))


def q8_1_offsets(M: int, K: int) -> dict:
    """Byte offsets of the sections of a q8_1 buffer (layout in include/mmq.h)."""
    kb = K // 32
    Mp = (M + 3) // 4 * 4
    ds = M * K
    h = (M * K + M * kb * 8 + 255) // 256 * 256
    dT = (h + 2 * M * K + 255) // 256 * 256
    return {"q": 0, "ds": ds, "h": h, "dT": dT, "sT": dT + Mp * kb * 4, "Mp": Mp}


def q8_1_views(buf: torch.Tensor, M: int, K: int):
    """(q int8 [M, K], ds f32 [M, K/32, 2]) views of a q8_1 buffer's block sections."""
    o = q8_1_offsets(M, K)
    q = buf[: M * K].view(torch.int8).view(M, K)
    ds = buf[o["ds"]: o["ds"] + M * (K // 32) * 8].view(torch.float32).view(M, K // 32, 2)
    return q, ds


def q8_1_shadow_views(buf: torch.Tensor, M: int, K: int):
    """(h fp16 [M, K], dT f32 [K/32, M], sT f32 [K/32, M]) views of a q8_1 buffer's derived sections."""
    o = q8_1_offsets(M, K)
    kb, Mp = K // 32, o["Mp"]
    h = buf[o["h"]: o["h"] + 2 * M * K].view(torch.float16).view(M, K)
    dT = buf[o["dT"]: o["dT"] + Mp * kb * 4].view(torch.float32).view(kb, Mp)[:, :M]
    sT = buf[o["sT"]: o["sT"] + Mp * kb * 4].view(torch.float32).view(kb, Mp)[:, :M]
    return h, dT, sT


def q8_1_prepare(buf: torch.Tensor, M: int, K: int, stream=None) -> torch.Tensor:
    """Fill the derived sections of a q8_1 buffer from its q and ds sections (mmq_q8_1_prepare)."""
    _check(load().mmq_q8_1_prepare(_ptr(buf), M, K, _stream(stream)), "mmq_q8_1_prepare")
    return buf


def pack_q8_1(q: torch.Tensor, d: torch.Tensor, s: torch.Tensor, device="cuda") -> torch.Tensor:
    """A complete q8_1 buffer on `device` from codes [M, K], scales d and block sums s [M, K/32]."""
    M, K = q.shape
    buf = torch.zeros(q8_1_bytes(M, K), dtype=torch.uint8, device=device)
    qv, dsv = q8_1_views(buf, M, K)
    qv.copy_(q.to(device))
    dsv.copy_(torch.stack([d.float(), s.float()], dim=-1).to(device))
    return q8_1_prepare(buf, M, K)


# ------------------------------------------------------------------------------------------ entry points
def quantize_q8_1(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x f32 [M, K] on the GPU -> q8_1 byte buffer (mmq_quantize_q8_1)."""
    M, K = x.shape
    if out is None:
        out = torch.empty(q8_1_bytes(M, K), dtype=torch.uint8, device=x.device)
    _check(load().mmq_quantize_q8_1(_ptr(x), M, K, _ptr(out), _stream(stream)), "mmq_quantize_q8_1")
    return out


def gemm(wtype: int, W: torch.Tensor, Xq: torch.Tensor, M: int, N: int, K: int, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Dense MMQ product (mmq_gemm): f32 [M, N] (bf16 for W8A8)."""
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16 if wtype == W8A8 else torch.float32, device=W.device)
    _check(load().mmq_gemm(wtype, _ptr(W), _ptr(Xq), _ptr(out), M, N, K, _stream(stream)), "mmq_gemm")
    return out


def gemm_debug_partials(wtype: int, W: torch.Tensor, Xq: torch.Tensor, M: int, N: int, K: int,
                        stream=None) -> torch.Tensor:
    """Exact per-group int32 dots (mmq_gemm_debug_partials): [M, N, K/G]."""
    G = 16 if wtype == IQ1_M else 32
    out = torch.empty((M, N, K // G), dtype=torch.int32, device=W.device)
    _check(load().mmq_gemm_debug_partials(wtype, _ptr(W), _ptr(Xq), _ptr(out), M, N, K, _stream(stream)),
           "mmq_gemm_debug_partials")
    return out


def gemm_debug_block_sums(wtype: int, W: torch.Tensor, Xq: torch.Tensor, M: int, N: int, K: int,
                          stream=None) -> torch.Tensor:
    """The TMA-fed kernel's exact 32-k block accumulators (mmq_gemm_debug_block_sums): int32 [M, N, K/32]."""
    out = torch.empty((M, N, K // 32), dtype=torch.int32, device=W.device)
    _check(load().mmq_gemm_debug_block_sums(wtype, _ptr(W), _ptr(Xq), _ptr(out), M, N, K, _stream(stream)),
           "mmq_gemm_debug_block_sums")
    return out


def gemm_id(wtype: int, W: torch.Tensor, n_experts: int, Xq: torch.Tensor, ids: torch.Tensor, M: int, N: int,
            K: int, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """MoE MUL_MAT_ID (mmq_gemm_id): f32 [M, slots, N]."""
    slots = ids.shape[1]
    if out is None:
        out = torch.empty((M, slots, N), dtype=torch.float32, device=W.device)
    need = gemm_id_workspace_bytes(M, K, slots, n_experts)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=W.device)
    _check(load().mmq_gemm_id(wtype, _ptr(W), n_experts, _ptr(Xq), _ptr(ids), slots, _ptr(out), M, N, K,
                              _ptr(workspace), workspace.numel(), _stream(stream)), "mmq_gemm_id")
    return out


def gemm_id_noalloc(wtype: int, W: torch.Tensor, n_experts: int, Xq: torch.Tensor, ids: torch.Tensor, M: int,
                    N: int, K: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """MoE MUL_MAT_ID without a workspace (mmq_gemm_id_noalloc): the routing lists live in the
    library's static device scratch array, for callers that cannot allocate device memory."""
    slots = ids.shape[1]
    if out is None:
        out = torch.empty((M, slots, N), dtype=torch.float32, device=W.device)
    _check(load().mmq_gemm_id_noalloc(wtype, _ptr(W), n_experts, _ptr(Xq), _ptr(ids), slots, _ptr(out), M, N, K,
                                      _stream(stream)), "mmq_gemm_id_noalloc")
    return out


def read_device_errors(stream=None) -> int:
    """Synchronise and return (and clear) the device error bits (DEVERR_*)."""
    bits = ctypes.c_uint(0)
    _check(load().mmq_read_device_errors(ctypes.byref(bits), _stream(stream)), "mmq_read_device_errors")
    return bits.value


def selftest_bounded_wait(device="cuda", stream=None) -> list[int]:
    """mmq_selftest_bounded_wait: [completed, abort_flag] of the polling and of the sleeping wait."""
    res = torch.full((4,), -1, dtype=torch.int32, device=device)
    _check(load().mmq_selftest_bounded_wait(_ptr(res), _stream(stream)), "mmq_selftest_bounded_wait")
    return res.cpu().tolist()


# ------------------------------------------------------------------------------- attention over the 8-bit cache
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class KVCache:
    """One layer's 8-bit paged cache (mmq_kv_cache): int8 codes k, v [pages, kv_heads, page_size, head_dim] and f32
    scales k_scale, v_scale [pages, kv_heads, page_size / block].  Holds the given tensors; nothing is copied."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "pages", "kv_heads", "page_size", "head_dim", "block", "_packed")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        shape, per = k.shape, k_scale.shape
        if k.dtype != torch.int8 or v.dtype != torch.int8 or v.shape != shape or len(shape) != 4:
            raise MMQError("KVCache: k and v are int8 tensors of one shape [pages, kv_heads, page_size, head_dim]")
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim = shape
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or v_scale.shape != per or \
                len(per) != 3 or per[0] != pages or per[1] != heads or not per[2] or page % per[2]:
            raise MMQError("KVCache: the scales are f32 tensors [pages, kv_heads, page_size / block]")
        self.block = page // per[2]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._packed = _CACHE.pack(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), pages, heads, dim, page, self.block)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page_size: int = 64, block: int = 16, device="cuda"):
        """A cache of unwritten pages (nothing has to be initialised)."""
        shape = (pages, kv_heads, page_size, head_dim)
        codes = [torch.empty(shape, dtype=torch.int8, device=device) for _ in range(2)]
        scales = [torch.empty((pages, kv_heads, page_size // block), dtype=torch.float32, device=device)
                  for _ in range(2)]
        return cls(*codes, *scales)


def _heads(t: torch.Tensor, what: str) -> bytes:
    dtype = _DTYPES.get(t.dtype)
    if dtype is None or not t.is_cuda or t.dim() != 3:
        raise MMQError(f"{what}: expected a CUDA tensor [tokens, heads, head_dim] of f32, bf16 or f16")
    ts, hs, ds = t.stride()
    if ds != 1:
        raise MMQError(f"{what}: the last dimension must be contiguous")
    return _HEADS.pack(t.data_ptr(), dtype, ts, hs)


def _typed(t: torch.Tensor | None, dtype, what: str) -> int | None:
    if t is None:
        return None
    if t.dtype is not dtype:
        raise MMQError(f"{what}: expected {dtype}")
    return _ptr(t)


def _vector(t: torch.Tensor | None, n: int, what: str) -> int | None:
    if t is None:
        return None
    if t.numel() != n:
        raise MMQError(f"{what}: expected {n} values")
    return _typed(t, torch.float32, what)


def _rotary(cos: torch.Tensor | None, sin: torch.Tensor | None, interleaved: bool) -> bytes | None:
    if cos is None and sin is None:
        return None
    if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape:
        raise MMQError("cos, sin: expected f32 tensors [positions, rot_dim / 2] of one shape")
    n, half = cos.shape
    return _ROTARY.pack(_typed(cos, torch.float32, "cos"), _typed(sin, torch.float32, "sin"), n, 2 * half,
                        1 if interleaved else 0)


def _seqs(page_table: torch.Tensor, kv_lens: torch.Tensor, cu_tokens: torch.Tensor | None) -> tuple[bytes, int]:
    n = kv_lens.numel()
    if page_table.dim() != 2 or page_table.shape[0] != n:
        raise MMQError("page_table: expected int32 [sequences, pages]")
    if cu_tokens is not None and cu_tokens.numel() != n + 1:
        raise MMQError("cu_tokens: expected int32 [sequences + 1]")
    return _SEQS.pack(_typed(page_table, torch.int32, "page_table"), page_table.shape[1],
                      _typed(kv_lens, torch.int32, "kv_lens"), _typed(cu_tokens, torch.int32, "cu_tokens") or 0, n), n


def _rows_out(like: torch.Tensor, out: torch.Tensor | None, dtype, what: str) -> torch.Tensor:
    if out is None:
        return torch.empty(like.shape, dtype=dtype or like.dtype, device=like.device)
    if out.shape != like.shape:
        raise MMQError(f"{what}: the output has another shape")
    return out


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                 cos: torch.Tensor | None = None, sin: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, dtype=None, stream=None):
    """RMS norm of query and key heads [tokens, heads, head_dim] and position rotation in one pass
    (mmq_qk_norm_rope): (q_out, k_out), of `dtype` (default: the inputs').  q_out = q works in place."""
    x = q if q is not None else k
    if x is None:
        raise MMQError("qk_norm_rope: neither q nor k given")
    T, _, D = x.shape
    if q is not None and k is not None and (k.shape[0] != T or k.shape[2] != D):
        raise MMQError("qk_norm_rope: q and k differ in tokens or head_dim")
    if positions is not None and positions.numel() != T:
        raise MMQError("qk_norm_rope: expected a position for each token")
    pq = pqo = pk = pko = None
    if q is not None:
        q_out = _rows_out(q, q_out, dtype, "qk_norm_rope")
        pq, pqo = _heads(q, "q"), _heads(q_out, "q_out")
    if k is not None:
        k_out = _rows_out(k, k_out, dtype, "qk_norm_rope")
        pk, pko = _heads(k, "k"), _heads(k_out, "k_out")
    rc = load().mmq_qk_norm_rope(pq, q.shape[1] if pq else 0, _vector(q_weight, D, "q_weight"), pqo,
                                 pk, k.shape[1] if pk else 0, _vector(k_weight, D, "k_weight"), pko, T, D,
                                 _typed(positions, torch.int32, "positions"), _rotary(cos, sin, interleaved), eps,
                                 _stream(stream))
    if rc:
        _check(rc, "mmq_qk_norm_rope")
    return q_out, k_out


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
              cu_tokens: torch.Tensor | None = None, cos: torch.Tensor | None = None, sin: torch.Tensor | None = None,
              interleaved: bool = False, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
              q: torch.Tensor | None = None, q_weight: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
              q_dtype=None, stream=None):
    """Quantize the new keys and values [tokens, kv_heads, head_dim] into the paged cache, normed and rotated on
    the way (mmq_kv_append).  kv_lens: cached tokens of each sequence, the new ones included.  Returns q_out (the
    queries normed and rotated in the same launch) where q is given."""
    T, H, D = k.shape
    if v.shape != k.shape or H != cache.kv_heads or D != cache.head_dim:
        raise MMQError("kv_append: k and v are [tokens, kv_heads, head_dim] of the cache")
    pq = pqo = None
    if q is not None:
        if q.shape[0] != T or q.shape[2] != D:
            raise MMQError("kv_append: q and k differ in tokens or head_dim")
        q_out = _rows_out(q, q_out, q_dtype, "kv_append")
        pq, pqo = _heads(q, "q"), _heads(q_out, "q_out")
    sq, _ = _seqs(page_table, kv_lens, cu_tokens)
    rc = load().mmq_kv_append(cache._packed, sq, T, _heads(k, "k"), _heads(v, "v"), _vector(k_weight, D, "k_weight"),
                              pq, q.shape[1] if pq else 0, _vector(q_weight, D, "q_weight"), pqo,
                              _rotary(cos, sin, interleaved), eps, _stream(stream))
    if rc:
        _check(rc, "mmq_kv_append")
    return q_out


def kv_read(cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor, tokens: int,
            cu_tokens: torch.Tensor | None = None, dtype=torch.bfloat16, stream=None):
    """The last cu_tokens[s+1] - cu_tokens[s] cached tokens of each sequence, `tokens` in all, as rows (k, v)
    [tokens, kv_heads, head_dim] of `dtype` (mmq_kv_read)."""
    shape, device = (tokens, cache.kv_heads, cache.head_dim), cache.k.device
    k, v = torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device)
    sq, _ = _seqs(page_table, kv_lens, cu_tokens)
    rc = load().mmq_kv_read(cache._packed, sq, tokens, _heads(k, "k"), _heads(v, "v"), _stream(stream))
    if rc:
        _check(rc, "mmq_kv_read")
    return k, v


def attention_workspace_bytes(tokens: int, heads: int, kv_heads: int, head_dim: int, seqs: int, max_tokens: int,
                              max_kv_len: int) -> int:
    return int(load().mmq_attention_workspace_bytes(tokens, heads, kv_heads, head_dim, seqs, max_tokens, max_kv_len))


def attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
              max_kv_len: int | None = None, cu_tokens: torch.Tensor | None = None, max_tokens: int | None = None,
              scale: float | None = None, causal: bool = True, window: int = 0, out: torch.Tensor | None = None,
              out_dtype=None, return_lse: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """softmax(scale q k^T) v over the 8-bit paged cache (mmq_attention): out [tokens, heads, head_dim], or
    (out, lse f32 [tokens, heads]).  max_kv_len and max_tokens bound a sequence's length and new tokens (default:
    what the page table holds; 1 without cu_tokens, else all tokens); scale defaults to head_dim ** -0.5."""
    T, H, D = q.shape
    if D != cache.head_dim:
        raise MMQError("attention: q has another head_dim than the cache")
    sq, seqs = _seqs(page_table, kv_lens, cu_tokens)
    if max_kv_len is None:
        max_kv_len = page_table.shape[1] * cache.page_size
    if max_tokens is None:
        max_tokens = 1 if cu_tokens is None else T
    out = _rows_out(q, out, out_dtype, "attention")
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if return_lse else None
    lib = load()
    if workspace is None:
        size = lib.mmq_attention_workspace_bytes(T, H, cache.kv_heads, D, seqs, max_tokens, max_kv_len)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    else:
        size = workspace.numel() * workspace.element_size()
    rc = lib.mmq_attention(_heads(q, "q"), H, cache._packed, sq, T, max_tokens, max_kv_len,
                           D ** -0.5 if scale is None else scale, 1 if causal else 0, window, _heads(out, "out"),
                           lse.data_ptr() if return_lse else None, _ptr(workspace), size, _stream(stream))
    if rc:
        _check(rc, "mmq_attention")
    return (out, lse) if return_lse else out
