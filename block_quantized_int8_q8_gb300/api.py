"""Thin Python binding of libmmq_gb300.so (argument marshalling only): ctypes, and for the attention operators, whose
calls are too short for that, a C++ module (bind/attention.cpp).

Every function forwards device pointers, sizes and the current CUDA stream to the C ABI declared in
include/mmq.h; all arithmetic runs in the library's sm_103a kernels.  PyTorch is used only for device
memory and streams.  If the library is missing or fails to load, every call raises: there is no CPU
fallback.

stream=: the stream to launch on (default: the current one).  Outputs and workspaces that a call makes come from
that stream's memory, as under torch.cuda.stream(stream); inputs have to be complete for it.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import operator
import os

import torch

from . import _build

Q8_0, Q4_0, Q4_K, IQ1_M, W8A8, Q6_K = 0, 1, 2, 3, 4, 5
DEVERR_TIMEOUT, DEVERR_EXPERT_ID, DEVERR_DUP_EXPERT = 1, 2, 4
DEVERR_PAGE, DEVERR_POSITION, DEVERR_LENGTH, DEVERR_DRAFT = 8, 16, 32, 64

#: every symbol include/mmq.h declares
EXPORTS = ("mmq_status_string", "mmq_last_cuda_error", "mmq_q8_1_bytes", "mmq_weight_bytes", "mmq_w8a8_act_bytes", "mmq_quantize_q8_1",
           "mmq_gemm", "mmq_gemm_id_workspace_bytes", "mmq_gemm_id", "mmq_gemm_debug_partials",
           "mmq_gemm_debug_block_sums", "mmq_selftest_bounded_wait",
           "mmq_read_device_errors", "mmq_gemm_id_noalloc", "mmq_q8_1_prepare",
           "mmq_qk_norm_rope", "mmq_kv_append", "mmq_kv_read", "mmq_attention_workspace_bytes", "mmq_attention",
           "mmq_draft_masks", "mmq_kv_append_tree", "mmq_attention_tree_workspace_bytes", "mmq_attention_tree",
           "mmq_kv_keep")
NOALLOC_SCRATCH_BYTES = 1 << 20

_lib = None
_bind = None


class MMQError(RuntimeError):
    pass


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
    F = ctypes.c_float                           # structures as P
    lib.mmq_qk_norm_rope.argtypes = [P, I, P, P, P, I, P, P, I64, I, P, P, F, P]
    lib.mmq_kv_append.argtypes = [P, P, I64, P, P, P, P, I, P, P, P, F, P]
    lib.mmq_kv_read.argtypes = [P, P, I64, P, P, P]
    lib.mmq_attention_workspace_bytes.argtypes = [I64, I, I, I, I, I64, I64]
    lib.mmq_attention_workspace_bytes.restype = SZ
    lib.mmq_attention.argtypes = [P, I, P, P, I64, I64, I64, F, I, I64, P, P, P, SZ, P]
    lib.mmq_draft_masks.argtypes = [P, P, I, I64, I64, P, P, I, P]
    lib.mmq_kv_append_tree.argtypes = [P, P, P, I64, P, P, P, P, I, P, P, P, F, P]
    lib.mmq_attention_tree_workspace_bytes.argtypes = [I64, I, I, I, I, I64, I64]
    lib.mmq_attention_tree_workspace_bytes.restype = SZ
    lib.mmq_attention_tree.argtypes = [P, I, P, P, P, I64, I64, I64, F, I64, P, P, P, SZ, P]
    lib.mmq_kv_keep.argtypes = [P, P, I64, P, I64, P, P]
    for f in (lib.mmq_qk_norm_rope, lib.mmq_kv_append, lib.mmq_kv_read, lib.mmq_attention, lib.mmq_draft_masks,
              lib.mmq_kv_append_tree, lib.mmq_attention_tree, lib.mmq_kv_keep):
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


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    # from the memory of the stream that writes it: the current stream may hand out again, or still read, its own
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


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
        out = _empty(q8_1_bytes(M, K), torch.uint8, x.device, stream)
    _check(load().mmq_quantize_q8_1(_ptr(x), M, K, _ptr(out), _stream(stream)), "mmq_quantize_q8_1")
    return out


def gemm(wtype: int, W: torch.Tensor, Xq: torch.Tensor, M: int, N: int, K: int, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Dense MMQ product (mmq_gemm): f32 [M, N] (bf16 for W8A8)."""
    if out is None:
        out = _empty((M, N), torch.bfloat16 if wtype == W8A8 else torch.float32, W.device, stream)
    _check(load().mmq_gemm(wtype, _ptr(W), _ptr(Xq), _ptr(out), M, N, K, _stream(stream)), "mmq_gemm")
    return out


def gemm_debug_partials(wtype: int, W: torch.Tensor, Xq: torch.Tensor, M: int, N: int, K: int,
                        stream=None) -> torch.Tensor:
    """Exact per-group int32 dots (mmq_gemm_debug_partials): [M, N, K/G]."""
    G = 16 if wtype == IQ1_M else 32
    out = _empty((M, N, K // G), torch.int32, W.device, stream)
    _check(load().mmq_gemm_debug_partials(wtype, _ptr(W), _ptr(Xq), _ptr(out), M, N, K, _stream(stream)),
           "mmq_gemm_debug_partials")
    return out


def gemm_debug_block_sums(wtype: int, W: torch.Tensor, Xq: torch.Tensor, M: int, N: int, K: int,
                          stream=None) -> torch.Tensor:
    """The TMA-fed kernel's exact 32-k block accumulators (mmq_gemm_debug_block_sums): int32 [M, N, K/32]."""
    out = _empty((M, N, K // 32), torch.int32, W.device, stream)
    _check(load().mmq_gemm_debug_block_sums(wtype, _ptr(W), _ptr(Xq), _ptr(out), M, N, K, _stream(stream)),
           "mmq_gemm_debug_block_sums")
    return out


def gemm_id(wtype: int, W: torch.Tensor, n_experts: int, Xq: torch.Tensor, ids: torch.Tensor, M: int, N: int,
            K: int, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """MoE MUL_MAT_ID (mmq_gemm_id): f32 [M, slots, N]."""
    slots = ids.shape[1]
    if out is None:
        out = _empty((M, slots, N), torch.float32, W.device, stream)
    need = gemm_id_workspace_bytes(M, K, slots, n_experts)
    if workspace is None:
        workspace = _empty(max(need, 16), torch.uint8, W.device, stream)
    _check(load().mmq_gemm_id(wtype, _ptr(W), n_experts, _ptr(Xq), _ptr(ids), slots, _ptr(out), M, N, K,
                              _ptr(workspace), workspace.numel(), _stream(stream)), "mmq_gemm_id")
    return out


def gemm_id_noalloc(wtype: int, W: torch.Tensor, n_experts: int, Xq: torch.Tensor, ids: torch.Tensor, M: int,
                    N: int, K: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """MoE MUL_MAT_ID without a workspace (mmq_gemm_id_noalloc): the routing lists live in the
    library's static device scratch array, for callers that cannot allocate device memory."""
    slots = ids.shape[1]
    if out is None:
        out = _empty((M, slots, N), torch.float32, W.device, stream)
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
    with torch.cuda.stream(stream):
        res = torch.full((4,), -1, dtype=torch.int32, device=device)
        _check(load().mmq_selftest_bounded_wait(_ptr(res), _stream(stream)), "mmq_selftest_bounded_wait")
        return res.cpu().tolist()


# ------------------------------------------------------------------------------- attention over the 8-bit cache
def _binding():
    """The C++ half of this binding (bind/attention.cpp), which marshals the calls below."""
    global _bind
    if _bind is None:
        load()
        path = _build.BIND_LIB
        if not os.path.exists(path):
            raise MMQError(f"binding not built: {path} is missing (run __graft_entry__.build())")
        loader = importlib.machinery.ExtensionFileLoader("_attention", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_attention", path, loader=loader))
        loader.exec_module(module)
        module.set_errors(MMQError, torch.OutOfMemoryError)
        _bind = module
    return _bind


class KVCache:
    """One layer's 8-bit paged cache (mmq_kv_cache): int8 codes k, v [pages, kv_heads, page_size, head_dim] and f32
    scales k_scale, v_scale [pages, kv_heads, page_size / block].  Holds the given tensors for good (the calls use
    their addresses as they are now); nothing is copied."""

    __slots__ = ("_k", "_v", "_k_scale", "_v_scale", "_pages", "_kv_heads", "_page_size", "_head_dim", "_block", "_packed")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        self._packed, self._pages, self._kv_heads, self._page_size, self._head_dim, self._block = \
            (_bind or _binding()).make_cache(k, v, k_scale, v_scale)
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale

    k, v, k_scale, v_scale, pages, kv_heads, page_size, head_dim, block = \
        (property(operator.attrgetter(name)) for name in __slots__[:-1])

    def __reduce__(self):                                     # a copy is a cache of the (copied) tensors
        return type(self), (self.k, self.v, self.k_scale, self.v_scale)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page_size: int = 64, block: int = 16, device="cuda"):
        """A cache of unwritten pages (nothing has to be initialised)."""
        if block <= 0 or page_size % block:
            raise MMQError(f"KVCache: page_size {page_size} is not a multiple of block {block}")
        shape = (pages, kv_heads, page_size, head_dim)
        codes = [torch.empty(shape, dtype=torch.int8, device=device) for _ in range(2)]
        scales = [torch.empty((pages, kv_heads, page_size // block), dtype=torch.float32, device=device)
                  for _ in range(2)]
        return cls(*codes, *scales)


def _handle(stream) -> int | None:
    return None if stream is None else stream.cuda_stream


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                 cos: torch.Tensor | None = None, sin: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, dtype=None, stream=None):
    """RMS norm of query and key heads [tokens, heads, head_dim] and position rotation in one pass
    (mmq_qk_norm_rope): (q_out, k_out), of `dtype` (default: the inputs').  q_out = q works in place."""
    return (_bind or _binding()).qk_norm_rope(q, k, positions, cos, sin, q_weight, k_weight, eps, interleaved, q_out,
                                              k_out, dtype, _handle(stream))


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
              cu_tokens: torch.Tensor | None = None, cos: torch.Tensor | None = None, sin: torch.Tensor | None = None,
              interleaved: bool = False, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
              q: torch.Tensor | None = None, q_weight: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
              q_dtype=None, stream=None, tree: "DraftTree | None" = None):
    """Quantize the new keys and values [tokens, kv_heads, head_dim] into the paged cache, normed and rotated on
    the way (mmq_kv_append).  kv_lens: cached tokens of each sequence, the new ones included.  Returns q_out (the
    queries normed and rotated in the same launch) where q is given.  With a tree of drafted tokens, keys and queries
    turn at the position of their depth and are stored in row order (mmq_kv_append_tree)."""
    depths, masks = _of_tree(tree)
    return (_bind or _binding()).kv_append(cache._packed, k, v, page_table, kv_lens, cu_tokens, cos, sin, interleaved,
                                           k_weight, eps, q, q_weight, q_out, q_dtype, _handle(stream), depths, masks)


def kv_read(cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor, tokens: int,
            cu_tokens: torch.Tensor | None = None, dtype=torch.bfloat16, stream=None):
    """The last cu_tokens[s+1] - cu_tokens[s] cached tokens of each sequence, `tokens` in all, as rows (k, v)
    [tokens, kv_heads, head_dim] of `dtype` (mmq_kv_read)."""
    return (_bind or _binding()).kv_read(cache._packed, cache._k, page_table, kv_lens, tokens, cu_tokens, dtype,
                                         _handle(stream))


def attention_workspace_bytes(tokens: int, heads: int, kv_heads: int, head_dim: int, seqs: int, max_tokens: int,
                              max_kv_len: int) -> int:
    return int(load().mmq_attention_workspace_bytes(tokens, heads, kv_heads, head_dim, seqs, max_tokens, max_kv_len))


def attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
              max_kv_len: int | None = None, cu_tokens: torch.Tensor | None = None, max_tokens: int | None = None,
              scale: float | None = None, causal: bool = True, window: int = 0, out: torch.Tensor | None = None,
              out_dtype=None, return_lse: bool = False, workspace: torch.Tensor | None = None, stream=None,
              tree: "DraftTree | None" = None):
    """softmax(scale q k^T) v over the 8-bit paged cache (mmq_attention): out [tokens, heads, head_dim], or
    (out, lse f32 [tokens, heads]).  max_kv_len and max_tokens bound a sequence's length and new tokens (default:
    what the page table holds; 1 without cu_tokens, else all tokens); scale defaults to head_dim ** -0.5.  With a tree of
    drafted tokens, a new token sees the cached ones before them all and, of the new, its ancestors and itself
    (mmq_attention_tree)."""
    depths, masks = _of_tree(tree)
    return (_bind or _binding()).attention(q, cache._packed, page_table, kv_lens, max_kv_len, cu_tokens, max_tokens,
                                           scale, causal, window, out, out_dtype, return_lse, workspace,
                                           _handle(stream), depths, masks)


# ------------------------------------------------------------------------------- a tree of drafted tokens
class DraftTree:
    """What the new tokens of a batch see of each other (mmq_draft_tree): depths int32 [tokens], the number of a token's
    ancestors, and masks int32 [tokens, words], bit j % 32 of word j / 32 set where it sees token j of its sequence.
    draft_tree() makes one from the tokens' parents, once for all layers."""

    __slots__ = ("depths", "masks")

    def __init__(self, depths: torch.Tensor, masks: torch.Tensor):
        self.depths, self.masks = depths, masks


def _of_tree(tree):
    if tree is None:
        return None, None
    if not isinstance(tree, DraftTree):
        raise MMQError("tree: expected a DraftTree")
    if tree.depths is None or tree.masks is None:             # (both None would pass for no tree)
        raise MMQError("tree: expected depths and masks")
    return tree.depths, tree.masks


def draft_tree(parents: torch.Tensor, cu_tokens: torch.Tensor | None = None, max_tokens: int | None = None,
               stream=None) -> DraftTree:
    """The tree (or trees) of each sequence's new tokens (mmq_draft_masks).  parents int32 [tokens]: the token that each
    one continues, counted within its sequence and before it, or -1 for the cached text.  max_tokens bounds a sequence's
    new tokens (default: 1 without cu_tokens, else all tokens), at most 1024."""
    return DraftTree(*(_bind or _binding()).draft_masks(parents, cu_tokens, max_tokens, _handle(stream)))


def attention_tree_workspace_bytes(tokens: int, heads: int, kv_heads: int, head_dim: int, seqs: int, max_tokens: int,
                                   max_kv_len: int) -> int:
    return int(load().mmq_attention_tree_workspace_bytes(tokens, heads, kv_heads, head_dim, seqs, max_tokens, max_kv_len))


def kv_keep(cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor, tokens: int, kept: torch.Tensor,
            counts: torch.Tensor, cu_tokens: torch.Tensor | None = None, stream=None) -> None:
    """Of each sequence's new tokens (`tokens` in all, the last of kv_lens), keep those of the rows kept[s, :counts[s]], which
    ascend, and move them up behind the cached text (mmq_kv_keep).  kept int32 [sequences, rows], counts int32
    [sequences].  The new lengths are kv_lens minus the new tokens plus counts."""
    (_bind or _binding()).kv_keep(cache._packed, page_table, kv_lens, tokens, kept, counts, cu_tokens, _handle(stream))
