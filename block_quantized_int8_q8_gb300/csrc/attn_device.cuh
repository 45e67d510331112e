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
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const __half* p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()));
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(__half* p, float x) { *p = __float2half_rn(x); }

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
// a THREADS-fold narrowing.
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
__device__ __forceinline__ void head_norm(float (&x0)[4], float (&x1)[4], const float (&w0)[4], const float (&w1)[4],
                                          float eps, bool on = true) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) s += x0[i] * x0[i] + x1[i] * x1[i];
    s = lane_sum<D / 8>(s);
    const float r = on ? rsqrtf(s * (1.0f / D) + eps) : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x0[i] = x0[i] * r * w0[i];
        x1[i] = x1[i] * r * w1[i];
    }
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float ra = a * c - b * s;
    b = a * s + b * c;
    a = ra;
}
__device__ __forceinline__ void head_turn(float (&x0)[4], float (&x1)[4], const float (&c)[4], const float (&s)[4],
                                          bool interleaved) {
    if (interleaved) {
        turn(x0[0], x0[1], c[0], s[0]);
        turn(x0[2], x0[3], c[1], s[1]);
        turn(x1[0], x1[1], c[2], s[2]);
        turn(x1[2], x1[3], c[3], s[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) turn(x0[i], x1[i], c[i], s[i]);
    }
}

}  // namespace mmq
