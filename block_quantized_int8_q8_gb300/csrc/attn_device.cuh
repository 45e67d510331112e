// attn_device.cuh -- device helpers shared by the attention operators: typed 4-element loads and stores,
// sequence lookup, head norm and position rotation.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "attn.h"
#include "mmq_device.cuh"

namespace mmq {

constexpr unsigned DEVERR_PAGE = 8u;
constexpr unsigned DEVERR_POSITION = 16u;
constexpr unsigned DEVERR_LENGTH = 32u;

__device__ __forceinline__ void flag_error(unsigned bit) { atomicOr(&g_mmq_device_errors, bit); }

// ------------------------------------------------------------------------------------------ typed rows
// Four neighbouring values as two packed f32 pairs: the arithmetic on rows is packed throughout, since these operators
// move so few bytes a value that plain instructions would bound them.
using Quad = uint64_t[2];

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// the bytes as loaded (half the registers while a load is in flight), and their values
template <typename T> struct RawOf { using type = uint2; };
template <> struct RawOf<float> { using type = uint4; };
template <typename T> using Raw = typename RawOf<T>::type;
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) { return *reinterpret_cast<const Raw<T>*>(p); }
__device__ __forceinline__ void expand(const uint4& v, Quad& x, float) {
    x[0] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void expand(const uint2& v, Quad& x, __nv_bfloat16) {
    x[0] = f2_pack(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
    x[1] = f2_pack(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ void expand(const uint2& v, Quad& x, __half) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    x[0] = f2_pack(a.x, a.y);
    x[1] = f2_pack(b.x, b.y);
}
__device__ __forceinline__ void load4(const float* p, Quad& x) { expand(load_raw(p), x, float()); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store4(float* p, const Quad& x) {
    *reinterpret_cast<float4*>(p) = make_float4(f2_lo(x[0]), f2_hi(x[0]), f2_lo(x[1]), f2_hi(x[1]));
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const Quad& x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f2_lo(x[0]), f2_hi(x[0]), T()), pack2(f2_lo(x[1]), f2_hi(x[1]), T()));
}

// launch_pdl with dynamic shared memory.
template <typename... Params, typename... Args>
inline cudaError_t launch_pdl_smem(void (*k)(Params...), dim3 grid, dim3 block, size_t bytes, cudaStream_t s,
                                   Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, static_cast<Params>(args)...);
}

// ------------------------------------------------------------------------------------------ sequences
// New tokens and length of a sequence, held within the packed rows and the page table.
struct Seq {
    int n0, n;                 // first packed row, new tokens
    int len;                   // cached tokens as stated
    int end;                   // tokens the page table can hold, at most len
};
// Offsets run from 0 to the number of tokens and do not fall: true where sequence s breaks that.
__device__ __forceinline__ bool odd_offsets(const SeqArgs& a, int s, int n0, int n1) {
    return n1 < n0 || (s == 0 && n0 != 0) || (s == a.seqs - 1 && n1 != a.tokens);
}
__device__ __forceinline__ Seq make_seq(const SeqArgs& a, int page, int n0, int n1, int len) {
    Seq q;
    q.n0 = max(n0, 0);
    q.n = max(min(n1, a.tokens) - q.n0, 0);
    q.len = max(len, 0);
    const long long cap = a.stride * page;
    q.end = (long long)q.len > cap ? (int)cap : q.len;
    return q;
}
__device__ __forceinline__ Seq load_seq(const SeqArgs& a, int s, int page) {
    return a.cu ? make_seq(a, page, a.cu[s], a.cu[s + 1], a.lens[s]) : make_seq(a, page, s, s + 1, a.lens[s]);
}

// The largest s with key(cu[s], s) <= x, for a non-decreasing key with key of 0 <= x, and that sequence; every thread of
// the block takes part.  Up to THREADS sequences in one round of loads, which brings the sequence's figures too; more by
// a THREADS-fold narrowing.  The grid's first block looks over all offsets on the way.
template <int THREADS, typename Key>
__device__ __forceinline__ int find_seq(const SeqArgs& a, int page, long long x, Key key, Seq& q) {
    __shared__ int s_seq[3];
    if (a.seqs <= THREADS) {
        const int i = threadIdx.x;
        int c0 = 0, c1 = 0, len = 0;
        if (i < a.seqs) {
            c0 = a.cu[i];
            c1 = a.cu[i + 1];
            len = a.lens[i];
            if (blockIdx.x == 0 && odd_offsets(a, i, c0, c1)) flag_error(DEVERR_LENGTH);
        }
        const int s = max(__syncthreads_count(i < a.seqs && key(c0, i) <= x) - 1, 0);
        if (i == s) {
            s_seq[0] = c0;
            s_seq[1] = c1;
            s_seq[2] = len;
        }
        __syncthreads();
        q = make_seq(a, page, s_seq[0], s_seq[1], s_seq[2]);
        return s;
    }
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.seqs; i += THREADS)
            if (odd_offsets(a, i, a.cu[i], a.cu[i + 1])) flag_error(DEVERR_LENGTH);
    int lo = 0, len = a.seqs;
    while (len > 1) {
        const int step = (len + THREADS - 1) / THREADS, at = (int)threadIdx.x * step;
        const int c = __syncthreads_count(at < len && key(a.cu[lo + at], lo + at) <= x);
        const int skip = max(c - 1, 0) * step;
        lo += skip;
        len = min(step, len - skip);
    }
    q = load_seq(a, lo, page);
    return lo;
}

// ------------------------------------------------------------------------------------------ norm and rotation
// A head of D values is held by D/8 neighbouring lanes, two chunks of four values each, so that a lane owns both
// values of its four rotation pairs: chunks at o0 and o1.  Pairs 4l .. 4l+3 belong to lane l; lanes past the
// rotated part hold the passed-through tail.
struct Chunks {
    int o0, o1;
    bool turn;
};
__device__ __forceinline__ Chunks head_chunks(int l, int half, bool interleaved) {
    Chunks c;
    c.turn = 4 * l < half;
    if (interleaved || half == 0) {
        c.o0 = 8 * l;
        c.o1 = c.o0 + 4;
    } else if (c.turn) {
        c.o0 = 4 * l;
        c.o1 = c.o0 + half;
    } else {
        c.o0 = 8 * l;          // 2*half + 2*(4l - half)
        c.o1 = c.o0 + 4;
    }
    return c;
}

template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// x / rms(x) * weight over the D values that D/8 lanes hold (unchanged where `on` is false; every lane takes part).
template <int D>
__device__ __forceinline__ void head_norm(Quad& x0, Quad& x1, const Quad& w0, const Quad& w1, float eps, bool on = true) {
    const uint64_t s2 = f2_fma(x1[1], x1[1], f2_fma(x1[0], x1[0], f2_fma(x0[1], x0[1], f2_mul(x0[0], x0[0]))));
    const float s = lane_sum<D / 8>(f2_lo(s2) + f2_hi(s2));
    const float r = on ? rsqrtf(s * (1.0f / D) + eps) : 1.0f;
    const uint64_t r2 = f2_pack(r, r);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        x0[i] = f2_mul(f2_mul(x0[i], r2), w0[i]);
        x1[i] = f2_mul(f2_mul(x1[i], r2), w1[i]);
    }
}

__device__ __forceinline__ uint64_t f2_neg(uint64_t v) { return v ^ 0x8000000080000000ull; }
// (a, b) -> (a c - b s, a s + b c) for the lane's four pairs
__device__ __forceinline__ void head_turn(Quad& x0, Quad& x1, const Quad& c, const Quad& s, bool interleaved) {
    if (interleaved) {
        // each packed pair is (a, b):  (a, b) c + (b, a) (-s, s)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint64_t& x = i < 2 ? x0[i] : x1[i - 2];
            const uint64_t cs = c[i >> 1], ss = s[i >> 1];
            const float ci = i & 1 ? f2_hi(cs) : f2_lo(cs), si = i & 1 ? f2_hi(ss) : f2_lo(ss);
            const uint64_t turned = f2_pack(f2_hi(x), f2_lo(x));
            x = f2_fma(x, f2_pack(ci, ci), f2_mul(turned, f2_pack(-si, si)));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint64_t a = x0[i], b = x1[i];
            x0[i] = f2_fma(a, c[i], f2_neg(f2_mul(b, s[i])));
            x1[i] = f2_fma(b, c[i], f2_mul(a, s[i]));
        }
    }
}

}  // namespace mmq
