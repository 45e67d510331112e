// attn_math.cuh -- arithmetic shared by the two attention kernels (attn_few.cu, attn_tiled.cu).
#pragma once
#include "attn_device.cuh"

namespace mmq {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float SCALE_FLOOR = 0x1p-64f;      // stands for a zero value scale (all codes zero) in log2 and 1/x
// A row's probabilities are 2^(t - m) with m, the reference, 2^HEAD below the largest term when it is set; a term may pass it
// by 2^LAZY before the sums are rescaled (fp16 ends just below 2^16: the rest is for the rounding of t, half a binary order
// where it is near 2^24).  Terms down to 2^-(HEAD + 14) of the largest then
// keep fp16's 11 bits and smaller ones are rounded to 2^-(HEAD + 25) of it, so that a long cache of weak terms beside
// a strong one is not lost: l sums the terms unrounded, and with HEAD 0 the 2^-25 of each made 4e-3 of the output at 131 k
// tokens.  What HEAD takes from the slack costs rescales: prompts 306 us with a slack of 12, 308 with 8, 321 with 4.
constexpr float HEAD = 7.f;
constexpr float LAZY = 15.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// word of four codes (c0..c3) -> fp16 pairs (c0, c2) and (c1, c3), exactly
__device__ __forceinline__ void codes_even_odd(uint32_t w, uint32_t& even, uint32_t& odd) {
    const uint32_t bias = 0x64806480u;                        // 1024 + 128
    const uint32_t e = (w & 0x00FF00FFu) ^ bias, o = ((w >> 8) & 0x00FF00FFu) ^ bias;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"(e), "r"(bias));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(o), "r"(bias));
}
__device__ __forceinline__ uint4 ld_cache(const int8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// The power of two that brings a row's largest magnitude m to [1, 2), and its inverse (0 and 0 for a zero row).  A
// bf16 row so scaled is exact in fp16 down to 2^-14 of its largest value and rounded to 2^-25 of it below.
__device__ __forceinline__ void row_scale(float m, float& up, float& down) {
    const int e = min(max((int)(__float_as_uint(m) >> 23), 1), 253);
    up = m == 0.f ? 0.f : __uint_as_float((unsigned)(254 - e) << 23);
    down = m == 0.f ? 0.f : __uint_as_float((unsigned)e << 23);
}
// eight bf16 or fp16 values -> f32
__device__ __forceinline__ void unpack8(const uint4& v, bool bf16, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (bf16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
// The part of the cache that a sequence's rows can see, in tiles of 16 tokens, and its parts of `chunk` tokens.
struct Range {
    int tile0, tiles, parts;
};
__device__ __forceinline__ Range visible_range(const AttnArgs& a, const Seq& q, int chunk) {
    const int n = min(q.n, a.max_tokens), end = min(q.end, a.max_kv), first = q.len - q.n;
    const int j0 = a.window > 0 ? max(first - a.window + 1, 0) : 0;
    const int j1 = a.causal ? min(end, first + n) : end;
    Range r;
    r.tile0 = j0 / 16;
    r.tiles = max((j1 + 15) / 16 - r.tile0, 0);
    r.parts = max((r.tiles * 16 + chunk - 1) / chunk, 1);
    return r;
}

}  // namespace mmq
