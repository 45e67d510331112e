// kv_cache.cu -- the operators that write and read the 8-bit paged key/value cache, and the head norm with the
// position rotation.
//
//   norm_rope  y = rotate(x / sqrt(mean x^2 + eps) * w), heads of D values
//   append     the same on the way into the cache, then per block of B tokens and head
//              s' = max(s, amax/127), code = round-half-even(x / s'); codes already there times s/s'
//   read       scale * code
//
// All of them move each value once.  Long calls are bound by memory bandwidth and by the instructions around each value
// (hence packed arithmetic, 16-byte or paired 8-byte accesses, no 64-bit divisions), short ones by the chain of dependent
// loads: sequence, page, rows.  GB300, each call over inputs larger than the last one left in the cache:
//   norm_rope  8191 tokens of 40 heads of 128, bf16: 30 us, 5.7 TB/s; 4 tokens: 2.5 us
//   append     6500 tokens of 32 query and 8 key/value heads, bf16: 34 us; 64 single tokens, f32: 6 us
//   read       131072 tokens of 8 heads to bf16: 132 us, 6.1 TB/s
#include "attn_device.cuh"
#include "internal.h"

namespace mmq {

namespace {

// ------------------------------------------------------------------------------------------ norm_rope
// A block takes `count` tokens; a group of D/8 lanes takes units of NR_HEADS heads of one token (their loads are in flight
// together; cos and sin are read once for them): queries first, then keys.
constexpr int NR_THREADS = 256;
constexpr int NR_HEADS = 4;

template <int D, typename TI, typename TO>
__global__ void __launch_bounds__(NR_THREADS, 4) norm_rope_kernel(const NormRopeArgs a, int count) {
    pdl_wait();
    constexpr int LANES = D / 8, GROUPS = NR_THREADS / LANES;
    const int uq = (a.q_heads + NR_HEADS - 1) / NR_HEADS, per = uq + (a.k_heads + NR_HEADS - 1) / NR_HEADS;
    const int t0 = blockIdx.x * count, units = min(count, a.tokens - t0) * per;
    const int l = threadIdx.x % LANES;
    const Chunks ch = head_chunks(l, a.rot.half, a.rot.interleaved);
    // groups of lanes go over the units together, so that every lane takes part in the sums
    for (int u0 = 0; u0 < units; u0 += GROUPS) {
        const int unit = u0 + threadIdx.x / LANES, j = min(unit / per, count - 1), u = unit - j * per, t = min(t0 + j, a.tokens - 1);
        const bool isq = u < uq;
        const int h0 = (isq ? u : u - uq) * NR_HEADS;
        int here = unit < units ? min((isq ? a.q_heads : a.k_heads) - h0, NR_HEADS) : 0;
        const int pos = a.rot.cos ? a.positions[t] : 0;
        const HeadRows in = isq ? a.q : a.k;
        const TI* src = static_cast<const TI*>(in.data) + t * in.ts + h0 * in.hs;
        Raw<TI> r0[NR_HEADS] = {}, r1[NR_HEADS] = {};
#pragma unroll
        for (int i = 0; i < NR_HEADS; i++) {
            if (i < here) {
                r0[i] = load_raw(src + ch.o0);
                r1[i] = load_raw(src + ch.o1);
            }
            src += in.hs;
        }
        Quad c, s;
        if (a.rot.cos && (pos < 0 || pos >= a.rot.positions)) {
            if (here > 0) flag_error(DEVERR_POSITION);
            here = 0;                                         // not written
        } else if (ch.turn) {
            load4(a.rot.cos + (long long)pos * a.rot.half + 4 * l, c);
            load4(a.rot.sin + (long long)pos * a.rot.half + 4 * l, s);
        }
        const float* weight = isq ? a.q_weight : a.k_weight;
        const bool norm = a.q_weight || a.k_weight;           // uniform: the lanes of a warp may hold both sides
        const uint64_t one = f2_pack(1.f, 1.f);
        Quad w0 = {one, one}, w1 = {one, one};
        if (weight) {
            load4(weight + ch.o0, w0);
            load4(weight + ch.o1, w1);
        }
        const HeadRows out = isq ? a.q_out : a.k_out;
        TO* dst = static_cast<TO*>(out.data) + t * out.ts + h0 * out.hs;
#pragma unroll
        for (int i = 0; i < NR_HEADS; i++) {
            Quad x0, x1;
            expand(r0[i], x0, TI());
            expand(r1[i], x1, TI());
            if (norm) head_norm<D>(x0, x1, w0, w1, a.eps, weight != nullptr);
            if (i < here) {
                if (ch.turn) head_turn(x0, x1, c, s, a.rot.interleaved);
                store4(dst + ch.o0, x0);
                store4(dst + ch.o1, x1);
            }
            dst += out.hs;
        }
    }
}

// ------------------------------------------------------------------------------------------ append
// One thread block per (block of B tokens, head, key or value): the rows of the block stay in registers between
// the largest magnitude and the codes, so the new rows are read once.  Other blocks take the queries; the two kinds are
// spread evenly over the grid, since one waits for memory more and the other works more (6500 tokens: 37 us with the
// queries last, 34 mixed).  A sequence of n new tokens touches at most n/B + 2 blocks, and at most n; slot
// cu[s]/B + 2s, or cu[s], is the first of sequence s (whichever makes fewer slots), so a block finds its sequence by a
// search and no list is built.
template <int D, int B> struct AppendShape {
    static constexpr int kLanes = D / 8;                    // lanes of one row
    // two rows a thread, within 128 to 512 threads
    static constexpr int kWant = B * kLanes / 2;
    static constexpr int kThreads = kWant < 128 ? 128 : (kWant > 512 ? 512 : kWant);
    static constexpr int kRows = kThreads / kLanes;         // rows of one pass
    static constexpr int kQHeads = 4;                       // query heads of one unit of a group of lanes
    static constexpr int kQTokens = 4;                      // most tokens of a block of queries
};

// The codes of four values for the scale d: round-half-even of the rounded quotients x/d.  t = x * inv, inv within 2 ulp
// of 1/d, lies within 4.6e-5 of the rounded quotient for |x/d| <= 127.5, and a rounding to integers only changes at
// half-integers: more than 1e-4 away from one, t rounds to the code; where one of the four is nearer, the quotients are
// formed.  Adding 1.5 * 2^23 rounds to an integer and leaves its low byte in place.
__device__ __forceinline__ uint32_t codes4(const Quad& x, float d, uint64_t inv2) {
    constexpr float MAGIC = 12582912.f;
    const uint64_t magic = f2_pack(MAGIC, MAGIC), unmagic = f2_pack(-MAGIC, -MAGIC);
    uint64_t y[2], off[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint64_t t = f2_mul(x[i], inv2);
        y[i] = f2_add(t, magic);
        off[i] = f2_add(t, f2_neg(f2_add(y[i], unmagic)));
    }
    const float far = fmaxf(fmaxf(fabsf(f2_lo(off[0])), fabsf(f2_hi(off[0]))),
                            fmaxf(fabsf(f2_lo(off[1])), fabsf(f2_hi(off[1]))));
    if (!(far <= 0.4999f)) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            y[i] = f2_pack(__fadd_rn(fminf(fmaxf(rintf(__fdiv_rn(f2_lo(x[i]), d)), -127.f), 127.f), MAGIC),
                           __fadd_rn(fminf(fmaxf(rintf(__fdiv_rn(f2_hi(x[i]), d)), -127.f), 127.f), MAGIC));
    }
    const uint32_t lo = __byte_perm((uint32_t)y[0], (uint32_t)(y[0] >> 32), 0x0040);
    const uint32_t hi = __byte_perm((uint32_t)y[1], (uint32_t)(y[1] >> 32), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ float largest(const Quad& x, float m) {
    m = fmaxf(m, fmaxf(fabsf(f2_lo(x[0])), fabsf(f2_hi(x[0]))));
    return fmaxf(m, fmaxf(fabsf(f2_lo(x[1])), fabsf(f2_hi(x[1]))));
}
__device__ __forceinline__ uint32_t scale_codes4(uint32_t w, float r) {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) o |= ((uint32_t)(int)rintf((float)(int8_t)(w >> (8 * i)) * r) & 0xFFu) << (8 * i);
    return o;
}

template <int D, int B, typename T>
__device__ __forceinline__ void append_block(const AppendArgs& a, int slot, int head, bool isv, bool by_token) {
    using S = AppendShape<D, B>;
    constexpr int NR = (B + S::kRows - 1) / S::kRows;
    int s = slot, local = 0;
    Seq q;
    if (a.sq.cu) {
        auto first = [=](int cu, int i) { return by_token ? (long long)cu : (long long)(cu / B) + 2ll * i; };
        s = find_seq<S::kThreads>(a.sq, a.c.page, slot, first, q);
        local = slot - (int)first(q.n0, s);
    } else {
        q = load_seq(a.sq, s, a.c.page);
    }
    if (q.n == 0 || local < 0) return;
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
    Raw<T> in0[NR] = {}, in1[NR] = {};
    bool fill[NR];
#pragma unroll
    for (int i = 0; i < NR; i++) {
        const int j = r0 + i * S::kRows, pos = b0 + j;
        fill[i] = j < B && pos >= p0 && pos < q.end;
        if (fill[i]) {
            const T* p = static_cast<const T*>(in.data) + (long long)(q.n0 + pos - p0) * in.ts + head * in.hs;
            in0[i] = load_raw(p + ch.o0);
            in1[i] = load_raw(p + ch.o1);
        }
    }
    Quad x0[NR], x1[NR];
#pragma unroll
    for (int i = 0; i < NR; i++) {
        expand(in0[i], x0[i], T());
        expand(in1[i], x1[i], T());
    }
    if (weight) {
        Quad w0, w1;
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
                x0[i][0] = x0[i][1] = x1[i][0] = x1[i][1] = 0ull;
            } else if (ch.turn) {
                Quad c, sn;
                load4(a.rot.cos + (long long)pos * a.rot.half + 4 * l, c);
                load4(a.rot.sin + (long long)pos * a.rot.half + 4 * l, sn);
                head_turn(x0[i], x1[i], c, sn, a.rot.interleaved);
            }
        }
        amax = largest(x1[i], largest(x0[i], amax));
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
    const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
    for (int i = 0; i < NR; i++) {
        const int j = r0 + i * S::kRows;
        uint32_t* p0w = reinterpret_cast<uint32_t*>(codes + j * D + ch.o0);
        uint32_t* p1w = reinterpret_cast<uint32_t*>(codes + j * D + ch.o1);
        if (fill[i]) {
            *p0w = d > 0.f ? codes4(x0[i], d, inv2) : 0u;
            *p1w = d > 0.f ? codes4(x1[i], d, inv2) : 0u;
        } else if (j < B && b0 + j < p0 && d != old) {
            const float r = __fdiv_rn(old, d);
            *p0w = scale_codes4(*p0w, r);
            *p1w = scale_codes4(*p1w, r);
        }
    }
}

// Queries of QTOKENS packed rows (one for a decode step, whose latency counts): positions first, then units of kQHeads
// heads of one token.
template <int D, int B, typename T>
__device__ __forceinline__ void append_queries(const AppendArgs& a, int t0, int count, int qot) {
    using S = AppendShape<D, B>;
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
    Quad w0, w1;
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
        Raw<T> r0[H] = {}, r1[H] = {};
#pragma unroll
        for (int i = 0; i < H; i++) {
            if (i < here) {
                r0[i] = load_raw(src + ch.o0);
                r1[i] = load_raw(src + ch.o1);
            }
            src += a.q.hs;
        }
        Quad c, sn;
        if (a.rot.cos && ch.turn && here > 0) {
            load4(a.rot.cos + (long long)pos * a.rot.half + 4 * l, c);
            load4(a.rot.sin + (long long)pos * a.rot.half + 4 * l, sn);
        }
        long long at = (long long)(t0 + j) * a.q_out.ts + h0 * a.q_out.hs;
#pragma unroll
        for (int i = 0; i < H; i++) {
            Quad x0, x1;
            expand(r0[i], x0, T());
            expand(r1[i], x1, T());
            if (a.q_weight) head_norm<D>(x0, x1, w0, w1, a.eps);
            if (i < here) {
                if (a.rot.cos && ch.turn) head_turn(x0, x1, c, sn, a.rot.interleaved);
                if (qot == MMQ_F32) {
                    store4(static_cast<float*>(a.q_out.data) + at + ch.o0, x0);
                    store4(static_cast<float*>(a.q_out.data) + at + ch.o1, x1);
                } else if (qot == MMQ_BF16) {
                    store4(static_cast<__nv_bfloat16*>(a.q_out.data) + at + ch.o0, x0);
                    store4(static_cast<__nv_bfloat16*>(a.q_out.data) + at + ch.o1, x1);
                } else {
                    store4(static_cast<__half*>(a.q_out.data) + at + ch.o0, x0);
                    store4(static_cast<__half*>(a.q_out.data) + at + ch.o1, x1);
                }
            }
            at += a.q_out.hs;
        }
    }
}

template <int D, int B, typename T>
__global__ void __launch_bounds__(AppendShape<D, B>::kThreads) append_kernel(const AppendArgs a, unsigned query_share,
                                                                          bool by_token, int qtokens, int qot) {
    pdl_wait();
    // block b is the q-th of the queries' where q grows at b, else one of the cache's
    const unsigned q = __umulhi(blockIdx.x, query_share), b = blockIdx.x - q;
    if (__umulhi(blockIdx.x + 1, query_share) == q) {
        const int slot = b / (2u * a.c.heads), w = b - slot * 2u * a.c.heads;
        const bool isv = w >= a.c.heads;
        append_block<D, B, T>(a, slot, isv ? w - a.c.heads : w, isv, by_token);
    } else {
        append_queries<D, B, T>(a, (int)q * qtokens, qtokens, qot);
    }
}

// ------------------------------------------------------------------------------------------ read
// One thread block per 8 packed rows, or as many as it has groups of lanes (f32 heads of 256: 4, with 128 threads 2); a group
// keeps one row and goes over its heads, a lane turns N codes into one 16-byte store.
// four codes -> f32 exactly: the byte spliced into the mantissa of 2^23 + x
__device__ __forceinline__ void codes_f32(uint32_t w, Quad& x) {
    const uint32_t u = w ^ 0x80808080u;
    const uint64_t bias = f2_pack(-8388736.f, -8388736.f);    // -(2^23 + 128)
    x[0] = f2_add(f2_pack(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)),
                          __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441))), bias);
    x[1] = f2_add(f2_pack(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)),
                          __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443))), bias);
}
__device__ __forceinline__ void store_codes(float* p, uint32_t w, uint64_t d2) {
    Quad x;
    codes_f32(w, x);
    x[0] = f2_mul(x[0], d2);
    x[1] = f2_mul(x[1], d2);
    store4(p, x);
}
template <typename T>
__device__ __forceinline__ void store_codes(T* p, uint2 w, uint64_t d2) {
    uint32_t o[4];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        Quad x;
        codes_f32(h ? w.y : w.x, x);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            x[i] = f2_mul(x[i], d2);
            o[2 * h + i] = pack2(f2_lo(x[i]), f2_hi(x[i]), T());
        }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
template <typename T> struct ReadVec { using type = uint2; static constexpr int n = 8; };
template <> struct ReadVec<float> { using type = uint32_t; static constexpr int n = 4; };

template <int D, typename T, int THREADS> struct ReadShape {
    static constexpr int kLanes = D / ReadVec<T>::n, kGroups = THREADS / kLanes;
    static constexpr int kTokens = kGroups < 8 ? kGroups : 8;
};

template <int D, typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) read_kernel(const ReadArgs a) {
    pdl_wait();
    using S = ReadShape<D, T, THREADS>;
    constexpr int N = ReadVec<T>::n;
    using V = typename ReadVec<T>::type;
    __shared__ long long s_page[S::kTokens];
    __shared__ int s_off[S::kTokens];
    const int t0 = blockIdx.x * S::kTokens;
    int s = t0;
    Seq q;
    if (a.sq.cu) s = find_seq<THREADS>(a.sq, a.c.page, t0, [](int cu, int) { return (long long)cu; }, q);
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
    // one side after the other; the group's heads a fixed distance apart in each
    constexpr int STEP = S::kGroups / S::kTokens;
    const int h0 = g / S::kTokens;
    const long long row = max(page, 0ll) * a.c.heads + h0;
    const long long code_step = (long long)STEP * a.c.page * D;
#pragma unroll
    for (int side = 0; side < 2; side++) {
        const HeadRows& o = side ? a.v_out : a.k_out;
        if (o.data == nullptr) continue;
        const int8_t* src = (side ? a.c.v : a.c.k) + (row * a.c.page + off) * D + N * l;
        const float* scale = (side ? a.c.vs : a.c.ks) + row * blocks + off / a.c.block;
        T* dst = static_cast<T*>(o.data) + (long long)(t0 + j) * o.ts + h0 * o.hs + N * l;
#pragma unroll 4
        for (int h = h0; h < a.c.heads; h += STEP) {
            V w{};
            float d = 0.f;
            if (page >= 0) {
                w = *reinterpret_cast<const V*>(src);
                d = *scale;
            }
            store_codes(dst, w, f2_pack(d, d));
            src += code_step;
            scale += STEP * blocks;
            dst += STEP * o.hs;
        }
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
    // one wave of blocks (8191 tokens: 31 us with 8 tokens a block, 33 with 4, 41 with 1)
    const int count = (a.tokens + 4 * 152 - 1) / (4 * 152);
    const unsigned grid = (unsigned)((a.tokens + (long long)count - 1) / count);
    return with_type(it, [&](auto ti) {
        return with_type(ot, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            return launch_pdl(norm_rope_kernel<D, TI, TO>, dim3(grid), dim3(NR_THREADS), s, a, count);
        });
    });
}

template <int D, int B>
cudaError_t launch_append(mmq_dtype t, mmq_dtype qot, const AppendArgs& a, cudaStream_t s) {
    using S = AppendShape<D, B>;
    const long long by_blocks = a.sq.tokens / B + 2ll * a.sq.seqs;
    const bool by_token = !a.sq.cu || a.sq.tokens <= by_blocks;      // (without offsets: one token for each sequence)
    const long long slots = by_token ? a.sq.tokens : by_blocks;
    const long long kv = slots * 2 * a.c.heads;
    // one token a block while that leaves SMs idle, else four
    const int qtokens = a.sq.tokens <= 8 * 152 ? 1 : S::kQTokens;
    const long long grid = kv + (a.q_heads > 0 ? ((long long)a.sq.tokens + qtokens - 1) / qtokens : 0);
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    // the queries' blocks for every 2^32 of the grid, rounded up: the last block's number comes out exactly
    const unsigned share = (unsigned)((((grid - kv) << 32) + grid - 1) / grid);
    return with_type(t, [&](auto ti) {
        return launch_pdl(append_kernel<D, B, decltype(ti)>, dim3((unsigned)grid), dim3(S::kThreads), s, a, share,
                          by_token, qtokens, (int)qot);
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

template <int D, typename T, int THREADS>
cudaError_t launch_read_threads(const ReadArgs& a, cudaStream_t s) {
    constexpr int tokens = ReadShape<D, T, THREADS>::kTokens;
    const unsigned grid = (unsigned)((a.sq.tokens + tokens - 1) / tokens);
    return launch_pdl(read_kernel<D, T, THREADS>, dim3(grid), dim3(THREADS), s, a);
}
// Many rows: smaller blocks, whose starts overlap other blocks' copies; few: more lanes on a row (131072 rows: 132 us
// with 128 threads, 154 with 256; an append of 6500 rows with their read: 52 us with 128, 49 with 256).
template <int D>
cudaError_t launch_read(mmq_dtype t, const ReadArgs& a, cudaStream_t s) {
    return with_type(t, [&](auto ti) {
        using T = decltype(ti);
        return a.sq.tokens > 32768 ? launch_read_threads<D, T, 128>(a, s) : launch_read_threads<D, T, 256>(a, s);
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
