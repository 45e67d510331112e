// kv_cache.cu -- the operators that write and read the 8-bit paged key/value cache, and the head norm with the
// position rotation.  All of them move each value once and are bound by memory bandwidth, or by launch latency for
// a decode step.
//
//   norm_rope  y = rotate(x / sqrt(mean x^2 + eps) * w), heads of D values
//   append     the same on the way into the cache, then per block of B tokens and head
//              s' = max(s, amax/127), code = round-half-even(x / s'); codes already there times s/s'
//   read       scale * code
#include "attn_device.cuh"
#include "internal.h"

namespace mmq {

namespace {

// ------------------------------------------------------------------------------------------ norm_rope
// One group of D/8 lanes takes HEADS heads of one token (their loads are in flight together; cos and sin are read
// once for them).  Queries first, then keys, in units of HEADS heads of one side.
constexpr int NR_THREADS = 256;
constexpr int NR_HEADS = 4;

template <int D, typename TI, typename TO>
__global__ void __launch_bounds__(NR_THREADS) norm_rope_kernel(const NormRopeArgs a) {
    pdl_wait();
    constexpr int LANES = D / 8, GROUPS = NR_THREADS / LANES;
    const int uq = (a.q_heads + NR_HEADS - 1) / NR_HEADS, uk = (a.k_heads + NR_HEADS - 1) / NR_HEADS;
    const long long unit = (long long)blockIdx.x * GROUPS + threadIdx.x / LANES;
    const long long t64 = unit / (uq + uk);
    const int u = (int)(unit - t64 * (uq + uk));
    const bool active = t64 < a.tokens;
    const int t = active ? (int)t64 : 0;
    const int l = threadIdx.x % LANES;
    const int pos = active && a.rot.cos ? a.positions[t] : 0;
    const Chunks ch = head_chunks(l, a.rot.half, a.rot.interleaved);
    const bool isq = u < uq;
    const int h0 = (isq ? u : u - uq) * NR_HEADS;
    int here = active ? min((isq ? a.q_heads : a.k_heads) - h0, NR_HEADS) : 0;
    const HeadRows in = isq ? a.q : a.k, out = isq ? a.q_out : a.k_out;
    const float* weight = isq ? a.q_weight : a.k_weight;
    const TI* src = static_cast<const TI*>(in.data) + t * in.ts + h0 * in.hs;
    TO* dst = static_cast<TO*>(out.data) + t * out.ts + h0 * out.hs;
    float x0[NR_HEADS][4], x1[NR_HEADS][4];
#pragma unroll
    for (int i = 0; i < NR_HEADS; i++) {
#pragma unroll
        for (int e = 0; e < 4; e++) x0[i][e] = x1[i][e] = 0.f;
        if (i < here) {
            load4(src + i * in.hs + ch.o0, x0[i]);
            load4(src + i * in.hs + ch.o1, x1[i]);
        }
    }
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.rot.cos && (pos < 0 || pos >= a.rot.positions)) {
        here = 0;                                             // not written
        flag_error(DEVERR_POSITION);
    } else if (active && ch.turn) {
        load4(a.rot.cos + (long long)pos * a.rot.half + 4 * l, c);
        load4(a.rot.sin + (long long)pos * a.rot.half + 4 * l, s);
    }
    if (a.q_weight || a.k_weight) {                          // uniform: the lanes of a warp may hold both sides
        float w0[4] = {1.f, 1.f, 1.f, 1.f}, w1[4] = {1.f, 1.f, 1.f, 1.f};
        if (weight) {
            load4(weight + ch.o0, w0);
            load4(weight + ch.o1, w1);
        }
#pragma unroll
        for (int i = 0; i < NR_HEADS; i++) head_norm<D>(x0[i], x1[i], w0, w1, a.eps, weight != nullptr);
    }
#pragma unroll
    for (int i = 0; i < NR_HEADS; i++) {
        if (ch.turn) head_turn(x0[i], x1[i], c, s, a.rot.interleaved);
        if (i < here) {
            store4(dst + i * out.hs + ch.o0, x0[i]);
            store4(dst + i * out.hs + ch.o1, x1[i]);
        }
    }
}

// ------------------------------------------------------------------------------------------ append
// One thread block per (block of B tokens, head, key or value): the rows of the block stay in registers between
// the largest magnitude and the codes, so the new rows are read once.  Blocks of the grid past those take the
// queries.  A sequence of n new tokens touches at most n/B + 2 blocks; slot cu[s]/B + 2s is the first of sequence s,
// so a block finds its sequence by a search and no list is built.
template <int D> struct AppendShape {
    static constexpr int kThreads = D == 256 ? 256 : 128;
    static constexpr int kLanes = D / 8;                    // lanes of one row
    static constexpr int kRows = kThreads / kLanes;         // rows of one pass: 16, 8, 8
    static constexpr int kQHeads = 4;                       // query heads of one unit of a group of lanes
    static constexpr int kQTokens = 8;                      // most tokens of a block of queries
};

// The code of x for the scale d, in the low byte: round-half-even of the rounded quotient x/d.  t = x * inv, inv within
// 2 ulp of 1/d, lies within 4.6e-5 of the rounded quotient for |x/d| <= 127.5, and a rounding to integers only
// changes at half-integers: more than 1e-4 away from one, t rounds to the code; nearer, the quotient is formed.  Adding
// 1.5 * 2^23 rounds to an integer and leaves its low bits in place.
__device__ __forceinline__ uint32_t code_byte(float x, float d, float inv) {
    constexpr float MAGIC = 12582912.f;
    const float t = __fmul_rn(x, inv);
    float y = __fadd_rn(t, MAGIC);
    if (!(fabsf(t - __fadd_rn(y, -MAGIC)) <= 0.4999f))
        y = __fadd_rn(fminf(fmaxf(rintf(__fdiv_rn(x, d)), -127.f), 127.f), MAGIC);
    return __float_as_uint(y);
}
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float d, float inv) {
    const uint32_t lo = __byte_perm(code_byte(x[0], d, inv), code_byte(x[1], d, inv), 0x0040);
    const uint32_t hi = __byte_perm(code_byte(x[2], d, inv), code_byte(x[3], d, inv), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ uint32_t scale_codes4(uint32_t w, float r) {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) o |= ((uint32_t)(int)rintf((float)(int8_t)(w >> (8 * i)) * r) & 0xFFu) << (8 * i);
    return o;
}

template <int D, int B, typename T>
__device__ __forceinline__ void append_block(const AppendArgs& a, int slot, int head, bool isv) {
    using S = AppendShape<D>;
    constexpr int NR = (B + S::kRows - 1) / S::kRows;
    int s = slot, local = 0;
    Seq q;
    if (a.sq.cu) {
        s = find_seq<S::kThreads>(a.sq, a.c.page, slot, [](int cu, int i) { return (long long)(cu / B) + 2ll * i; }, q);
        local = slot - (q.n0 / B + 2 * s);
    } else {
        q = load_seq(a.sq, s, a.c.page);
    }
    if (q.n == 0) return;
    const int p0 = q.len - q.n;                              // position of the first new token
    if (threadIdx.x == 0 && local == 0 && (p0 < 0 || q.end < q.len)) flag_error(DEVERR_LENGTH);
    const int b0 = (max(p0, 0) / B + local) * B;             // first position of this block
    if (b0 >= q.end) return;
    const int pg = a.sq.table[s * a.sq.stride + b0 / a.c.page];
    if ((unsigned)pg >= (unsigned long long)a.c.pages) {
        if (threadIdx.x == 0) flag_error(DEVERR_PAGE);
        return;
    }
    const int off = b0 % a.c.page;
    const long long ph = (long long)pg * a.c.heads + head;
    int8_t* codes = (isv ? a.c.v : a.c.k) + (ph * a.c.page + off) * D;
    float* scale = (isv ? a.c.vs : a.c.ks) + ph * (a.c.page / B) + off / B;
    const bool fresh = p0 <= b0;
    const float old = fresh ? 0.f : *scale;

    const HeadRows& in = isv ? a.v : a.k;
    const bool rotate = !isv && a.rot.cos != nullptr;
    const float* weight = isv ? nullptr : a.k_weight;
    const int l = threadIdx.x % S::kLanes, r0 = threadIdx.x / S::kLanes;
    const Chunks ch = head_chunks(l, rotate ? a.rot.half : 0, a.rot.interleaved);
    float x0[NR][4], x1[NR][4];
    bool fill[NR];
#pragma unroll
    for (int i = 0; i < NR; i++) {
        const int j = r0 + i * S::kRows, pos = b0 + j;
        fill[i] = j < B && pos >= p0 && pos < q.end;
#pragma unroll
        for (int e = 0; e < 4; e++) x0[i][e] = x1[i][e] = 0.f;
        if (fill[i]) {
            const T* p = static_cast<const T*>(in.data) + (long long)(q.n0 + pos - p0) * in.ts + head * in.hs;
            load4(p + ch.o0, x0[i]);
            load4(p + ch.o1, x1[i]);
        }
    }
    if (weight) {
        float w0[4], w1[4];
        load4(weight + ch.o0, w0);
        load4(weight + ch.o1, w1);
#pragma unroll
        for (int i = 0; i < NR; i++) head_norm<D>(x0[i], x1[i], w0, w1, a.eps);
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < NR; i++) {
        const int pos = b0 + r0 + i * S::kRows;
        if (rotate && fill[i]) {
            if (pos >= a.rot.positions) {
                fill[i] = false;
                if (l == 0) flag_error(DEVERR_POSITION);
#pragma unroll
                for (int e = 0; e < 4; e++) x0[i][e] = x1[i][e] = 0.f;
            } else if (ch.turn) {
                float c[4], sn[4];
                load4(a.rot.cos + (long long)pos * a.rot.half + 4 * l, c);
                load4(a.rot.sin + (long long)pos * a.rot.half + 4 * l, sn);
                head_turn(x0[i], x1[i], c, sn, a.rot.interleaved);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e++) amax = fmaxf(amax, fmaxf(fabsf(x0[i][e]), fabsf(x1[i][e])));
    }
    // block-wide largest magnitude (the bits of non-negative floats order as integers)
    __shared__ unsigned s_amax[S::kThreads / 32];
    const unsigned wmax = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
    if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = wmax;
    __syncthreads();
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < S::kThreads / 32; i++) m = max(m, s_amax[i]);
    float need = __fdiv_rn(__uint_as_float(m), 127.f);
    if (need < 0x1p-63f) need = 0.f;
    const float d = fmaxf(old, need);
    if (threadIdx.x == 0 && (fresh || d != old)) *scale = d;
    const float inv = __fdividef(1.f, d);
#pragma unroll
    for (int i = 0; i < NR; i++) {
        const int j = r0 + i * S::kRows;
        uint32_t* p0w = reinterpret_cast<uint32_t*>(codes + j * D + ch.o0);
        uint32_t* p1w = reinterpret_cast<uint32_t*>(codes + j * D + ch.o1);
        if (fill[i]) {
            *p0w = d > 0.f ? codes4(x0[i], d, inv) : 0u;
            *p1w = d > 0.f ? codes4(x1[i], d, inv) : 0u;
        } else if (j < B && b0 + j < p0 && d != old) {
            const float r = __fdiv_rn(old, d);
            *p0w = scale_codes4(*p0w, r);
            *p1w = scale_codes4(*p1w, r);
        }
    }
}

// Queries of QTOKENS packed rows (one for a decode step, whose latency counts): positions first, then units of kQHeads
// heads of one token.
template <int D, typename T>
__device__ __forceinline__ void append_queries(const AppendArgs& a, int t0, int count, int qot) {
    using S = AppendShape<D>;
    constexpr int H = S::kQHeads;
    __shared__ int s_pos[S::kQTokens];
    Seq q;
    int s = t0;
    if (a.sq.cu) s = find_seq<S::kThreads>(a.sq, a.c.page, t0, [](int cu, int) { return (long long)cu; }, q);
    if (threadIdx.x < count) {
        const int t = t0 + threadIdx.x;
        int pos = -1;
        if (t < a.sq.tokens) {
            if (!a.sq.cu) {
                q = load_seq(a.sq, t, a.c.page);
            } else if (t >= q.n0 + q.n) {
                while (s + 1 < a.sq.seqs && a.sq.cu[s + 1] <= t) s++;
                q = load_seq(a.sq, s, a.c.page);
            }
            if (t >= q.n0 && t < q.n0 + q.n) pos = q.len - q.n + (t - q.n0);
            if (a.rot.cos && pos >= a.rot.positions) {
                pos = -1;
                flag_error(DEVERR_POSITION);
            }
        }
        s_pos[threadIdx.x] = pos;
    }
    __syncthreads();
    const int per = (a.q_heads + H - 1) / H, l = threadIdx.x % S::kLanes;
    const Chunks ch = head_chunks(l, a.rot.cos ? a.rot.half : 0, a.rot.interleaved);
    float w0[4], w1[4];
    if (a.q_weight) {
        load4(a.q_weight + ch.o0, w0);
        load4(a.q_weight + ch.o1, w1);
    }
    // groups of lanes go over the units together, so that every lane takes part in the sums
    for (int u0 = 0; u0 < count * per; u0 += S::kRows) {
        const int u = u0 + threadIdx.x / S::kLanes, j = min(u / per, count - 1), h0 = (u - j * per) * H;
        const int pos = u < count * per ? s_pos[j] : -1;
        const int here = pos < 0 ? 0 : min(a.q_heads - h0, H);
        const T* src = static_cast<const T*>(a.q.data) + (long long)(t0 + j) * a.q.ts + h0 * a.q.hs;
        float x0[H][4], x1[H][4], c[4], sn[4];
#pragma unroll
        for (int i = 0; i < H; i++) {
#pragma unroll
            for (int e = 0; e < 4; e++) x0[i][e] = x1[i][e] = 0.f;
            if (i < here) {
                load4(src + i * a.q.hs + ch.o0, x0[i]);
                load4(src + i * a.q.hs + ch.o1, x1[i]);
            }
        }
        if (a.rot.cos && ch.turn && here > 0) {
            load4(a.rot.cos + (long long)pos * a.rot.half + 4 * l, c);
            load4(a.rot.sin + (long long)pos * a.rot.half + 4 * l, sn);
        }
        if (a.q_weight) {
#pragma unroll
            for (int i = 0; i < H; i++) head_norm<D>(x0[i], x1[i], w0, w1, a.eps);
        }
#pragma unroll
        for (int i = 0; i < H; i++) {
            if (i >= here) break;
            if (a.rot.cos && ch.turn) head_turn(x0[i], x1[i], c, sn, a.rot.interleaved);
            const long long at = (long long)(t0 + j) * a.q_out.ts + (h0 + i) * a.q_out.hs;
            if (qot == MMQ_F32) {
                store4(static_cast<float*>(a.q_out.data) + at + ch.o0, x0[i]);
                store4(static_cast<float*>(a.q_out.data) + at + ch.o1, x1[i]);
            } else if (qot == MMQ_BF16) {
                store4(static_cast<__nv_bfloat16*>(a.q_out.data) + at + ch.o0, x0[i]);
                store4(static_cast<__nv_bfloat16*>(a.q_out.data) + at + ch.o1, x1[i]);
            } else {
                store4(static_cast<__half*>(a.q_out.data) + at + ch.o0, x0[i]);
                store4(static_cast<__half*>(a.q_out.data) + at + ch.o1, x1[i]);
            }
        }
    }
}

template <int D, int B, typename T>
__global__ void __launch_bounds__(AppendShape<D>::kThreads) append_kernel(const AppendArgs a, long long kv_blocks,
                                                                          int qtokens, int qot) {
    pdl_wait();
    const long long b = blockIdx.x;
    if (b < kv_blocks) {
        const int slot = (int)(b / (2 * a.c.heads)), w = (int)(b - (long long)slot * 2 * a.c.heads);
        const bool isv = w >= a.c.heads;
        append_block<D, B, T>(a, slot, isv ? w - a.c.heads : w, isv);
    } else {
        append_queries<D, T>(a, (int)(b - kv_blocks) * qtokens, qtokens, qot);
    }
}

// ------------------------------------------------------------------------------------------ read
// One thread block per 8 packed rows (4 of the widest f32 heads); a group of lanes keeps one row and goes over its heads,
// a lane turns N codes into one 16-byte store.
constexpr int READ_THREADS = 256;

__device__ __forceinline__ void store_codes(float* p, uint32_t w, float d) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; i++) x[i] = (float)(int8_t)(w >> (8 * i)) * d;
    store4(p, x);
}
template <typename T>
__device__ __forceinline__ void store_codes(T* p, uint2 w, float d) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[i] = (float)(int8_t)(w.x >> (8 * i)) * d;
        x[4 + i] = (float)(int8_t)(w.y >> (8 * i)) * d;
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()), pack2(x[4], x[5], T()),
                                              pack2(x[6], x[7], T()));
}
template <typename T> struct ReadVec { using type = uint2; static constexpr int n = 8; };
template <> struct ReadVec<float> { using type = uint32_t; static constexpr int n = 4; };

template <int D, typename T> struct ReadShape {
    static constexpr int kLanes = D / ReadVec<T>::n, kGroups = READ_THREADS / kLanes;
    static constexpr int kTokens = kGroups < 8 ? kGroups : 8;
};

template <int D, typename T>
__global__ void __launch_bounds__(READ_THREADS) read_kernel(const ReadArgs a) {
    pdl_wait();
    using S = ReadShape<D, T>;
    constexpr int N = ReadVec<T>::n;
    using V = typename ReadVec<T>::type;
    __shared__ long long s_page[S::kTokens];
    __shared__ int s_off[S::kTokens];
    const int t0 = blockIdx.x * S::kTokens;
    int s = t0;
    Seq q;
    if (a.sq.cu) s = find_seq<READ_THREADS>(a.sq, a.c.page, t0, [](int cu, int) { return (long long)cu; }, q);
    if (threadIdx.x < S::kTokens) {
        const int t = t0 + threadIdx.x;
        long long page = -2;                                 // past the rows
        int off = 0;
        if (t < a.sq.tokens) {
            if (!a.sq.cu) {
                s = t;
                q = load_seq(a.sq, t, a.c.page);
            } else if (t >= q.n0 + q.n) {
                while (s + 1 < a.sq.seqs && a.sq.cu[s + 1] <= t) s++;
                q = load_seq(a.sq, s, a.c.page);
            }
            const int pos = q.len - q.n + (t - q.n0);
            page = -1;                                       // a row of zeros
            if (t >= q.n0 && t < q.n0 + q.n && pos >= 0 && pos < q.end) {
                page = a.sq.table[s * a.sq.stride + pos / a.c.page];
                off = pos % a.c.page;
                if (page < 0 || page >= a.c.pages) {
                    page = -1;
                    flag_error(DEVERR_PAGE);
                }
            } else {
                flag_error(DEVERR_LENGTH);
            }
        }
        s_page[threadIdx.x] = page;
        s_off[threadIdx.x] = off;
    }
    __syncthreads();
    const int l = threadIdx.x % S::kLanes, g = threadIdx.x / S::kLanes, j = g % S::kTokens;
    const long long page = s_page[j];
    if (page == -2) return;
    const int off = s_off[j], blocks = a.c.page / a.c.block;
    const long long row0 = max(page, 0ll) * a.c.heads, code0 = (long long)off * D + N * l;
    // units: key heads, then value heads
    const bool hk = a.k_out.data != nullptr, hv = a.v_out.data != nullptr;
    const int first = hk ? 0 : a.c.heads, units = hv ? 2 * a.c.heads : a.c.heads;
#pragma unroll 8
    for (int u = first + g / S::kTokens; u < units; u += S::kGroups / S::kTokens) {
        const bool isv = u >= a.c.heads;
        const int head = isv ? u - a.c.heads : u;
        V w{};
        float d = 0.f;
        if (page >= 0) {
            w = *reinterpret_cast<const V*>((isv ? a.c.v : a.c.k) + (row0 + head) * a.c.page * D + code0);
            d = (isv ? a.c.vs : a.c.ks)[(row0 + head) * blocks + off / a.c.block];
        }
        const HeadRows& o = isv ? a.v_out : a.k_out;
        store_codes(static_cast<T*>(o.data) + (long long)(t0 + j) * o.ts + head * o.hs + N * l, w, d);
    }
}

// ------------------------------------------------------------------------------------------ launches
template <typename F>
cudaError_t with_type(mmq_dtype t, F f) {
    switch (t) {
        case MMQ_F32: return f(float());
        case MMQ_BF16: return f(__nv_bfloat16());
        case MMQ_F16: return f(__half());
    }
    return cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_norm_rope(mmq_dtype it, mmq_dtype ot, const NormRopeArgs& a, cudaStream_t s) {
    constexpr int GROUPS = NR_THREADS / (D / 8);
    const long long units = (long long)a.tokens *
                            ((a.q_heads + NR_HEADS - 1) / NR_HEADS + (a.k_heads + NR_HEADS - 1) / NR_HEADS);
    const long long grid = (units + GROUPS - 1) / GROUPS;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    return with_type(it, [&](auto ti) {
        return with_type(ot, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            return launch_pdl(norm_rope_kernel<D, TI, TO>, dim3((unsigned)grid), dim3(NR_THREADS), s, a);
        });
    });
}

template <int D, int B>
cudaError_t launch_append(mmq_dtype t, mmq_dtype qot, const AppendArgs& a, cudaStream_t s) {
    using S = AppendShape<D>;
    const long long slots = a.sq.cu ? a.sq.tokens / B + 2ll * a.sq.seqs : a.sq.seqs;
    const long long kv = slots * 2 * a.c.heads;
    // one token a block while that leaves SMs idle, else eight
    const int qtokens = a.sq.tokens <= 8 * 152 ? 1 : S::kQTokens;
    const long long grid = kv + (a.q_heads > 0 ? ((long long)a.sq.tokens + qtokens - 1) / qtokens : 0);
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    return with_type(t, [&](auto ti) {
        return launch_pdl(append_kernel<D, B, decltype(ti)>, dim3((unsigned)grid), dim3(S::kThreads), s, a, kv,
                          qtokens, (int)qot);
    });
}

template <int D>
cudaError_t launch_append_block(mmq_dtype t, mmq_dtype qot, const AppendArgs& a, cudaStream_t s) {
    switch (a.c.block) {
        case 16: return launch_append<D, 16>(t, qot, a, s);
        case 32: return launch_append<D, 32>(t, qot, a, s);
        case 64: return launch_append<D, 64>(t, qot, a, s);
    }
    return cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_read(mmq_dtype t, const ReadArgs& a, cudaStream_t s) {
    return with_type(t, [&](auto ti) {
        constexpr int tokens = ReadShape<D, decltype(ti)>::kTokens;
        const unsigned grid = (unsigned)((a.sq.tokens + tokens - 1) / tokens);
        return launch_pdl(read_kernel<D, decltype(ti)>, dim3(grid), dim3(READ_THREADS), s, a);
    });
}

}  // namespace

cudaError_t run_norm_rope(int dim, mmq_dtype it, mmq_dtype ot, const NormRopeArgs& a, cudaStream_t s) {
    switch (dim) {
        case 64: return launch_norm_rope<64>(it, ot, a, s);
        case 128: return launch_norm_rope<128>(it, ot, a, s);
        case 256: return launch_norm_rope<256>(it, ot, a, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t run_kv_append(int dim, mmq_dtype t, mmq_dtype qot, const AppendArgs& a, cudaStream_t s) {
    switch (dim) {
        case 64: return launch_append_block<64>(t, qot, a, s);
        case 128: return launch_append_block<128>(t, qot, a, s);
        case 256: return launch_append_block<256>(t, qot, a, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t run_kv_read(int dim, mmq_dtype t, const ReadArgs& a, cudaStream_t s) {
    switch (dim) {
        case 64: return launch_read<64>(t, a, s);
        case 128: return launch_read<128>(t, a, s);
        case 256: return launch_read<256>(t, a, s);
    }
    return cudaErrorInvalidValue;
}

MMQ_DEFINE_ERROR_READER(kv_cache)

}  // namespace mmq
