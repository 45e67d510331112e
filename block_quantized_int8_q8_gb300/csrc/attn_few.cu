// attn_few.cu -- attention of few query rows over the 8-bit paged cache: single new tokens (decode) and the few of a
// verification step, up to 16 rows (new tokens x query heads) for each sequence and key/value head.
//
//   t_j = scale log2(e) ks_b (q . k_j) + log2(vs_b)      k_j, v_j: int8 codes, b the block of token j
//   p_j = 2^(t_j - m),  O = sum_j p_j v_j,  l = sum_b (1/vs_b) sum_{j in b} p_j,  out = O / l,
//   lse = ln(2) (m + log2 l)
// The value scale enters the exponent, so that it costs nothing per value and the fp16 probabilities stay relative
// to the largest term; O and l are f32.
//
// Bound by reading the cache, closely followed by the integer instructions that turn codes into fp16 (a lane spends 5 on
// four codes).  Each warp walks tiles of 16 tokens of its own (head_dim 64: two at a time): asynchronous 16-byte copies
// into a ring in shared memory, two steps ahead, then reads straight into tensor-core fragments.  The product
// S^T = K Q^T has 16 tokens as rows and 8 query rows as columns, so a group of up to 8 query heads wastes nothing, and
// O^T = V^T P^T takes P^T from S^T by a transposing register move.  Which head dimension a fragment element means is free
// as long as both operands agree, so K rows are read as quarters of 64 bytes and V through transposed reads of byte
// pairs; the copies permute each row's 16-byte chunks so that neither read meets a bank twice.  int8 -> fp16 is exact
// (byte spliced into the mantissa of 1024 + x).  The cache range is split over thread blocks in chunks; each thread
// block joins its four warps in shared memory, a second launch joins the chunks.
// GB300, heads of 128, 32 query and 8 key/value heads: 64 sequences of up to 8192 tokens 101 us (5.4 TB/s of cache), of
// which the join takes 6; one sequence of 131 k tokens 54 us (5.0 TB/s), the join 5; one of 77 tokens 4.6 us.  With the
// tiles loaded straight into registers a tile ahead the first two took 114 and 59 us; with V through byte shuffles 105 and
// 60; chunks of 1024 or 4096 tokens instead of 2048 for the batch: 100 and 113 us; parts joined through the shared memory of
// a cluster instead of by a second launch: 107 (its blocks hold their places until the last has finished).
#include "attn_device.cuh"
#include "attn_math.cuh"
#include "internal.h"

namespace mmq {

namespace {

constexpr int FEW_WARPS = 4;
constexpr int FEW_THREADS = FEW_WARPS * 32;
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Pitch of a row of partial sums in shared memory: a fragment's 8-byte stores (columns 2t, dimensions 2g) fall on
// different banks.
template <int D> constexpr int kSumPitch = D + 4;

// Shared memory: fp16 queries, the warps' rings, and over these at the end the warps' sums.
template <int D, int NT> struct FewSmem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kStep = D == 64 ? 2 : 1;                                    // tiles of 16 tokens taken at once
    static constexpr int kStages = 3;                                                // 12 KB a warp (head_dim 256: 24)
    static constexpr int kTile = 16 * D;                                             // bytes of a tile's K or V
    static constexpr int kScale = kRows * (D + 8) * 2;
    static constexpr int kRing = kScale + FEW_WARPS * kStages * kStep * 16;
    static constexpr int kBytes = kRing + FEW_WARPS * kStages * kStep * 2 * kTile;
    static_assert(FEW_WARPS * kRows * kSumPitch<D> * 4 <= kBytes - kRing, "the sums fit over the rings");
};

// Where 16-byte chunk c of row r of a tile lies.  K is read as four neighbouring chunks of rows 2i, 2i+1 at a time, V as
// one chunk of eight rows.
template <int D> __device__ __forceinline__ int k_at(int r, int c) {
    return D == 64 ? r * 64 + c * 16 : r * D + ((c ^ ((r & 1) << 2)) << 4);
}
template <int D> __device__ __forceinline__ int v_at(int r, int c) {
    return D == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * D + ((c ^ (r & 7)) << 4);
}

// Four 8 x 16-byte matrices, transposed in 2-byte units: register i of lane (g, t) holds bytes 2g, 2g+1 of rows 2t and 2t+1
// of matrix i, whose row r is at lane 8i + r's address.
__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void store_out4(void* p, long long at, const float (&x)[4], int type) {
    const Quad v = {f2_pack(x[0], x[1]), f2_pack(x[2], x[3])};
    if (type == MMQ_F32) store4(static_cast<float*>(p) + at, v);
    else if (type == MMQ_BF16) store4(static_cast<__nv_bfloat16*>(p) + at, v);
    else store4(static_cast<__half*>(p) + at, v);
}

template <int D, int NT>
__global__ void __launch_bounds__(FEW_THREADS, few_blocks(D, NT)) few_kernel(const AttnArgs a, int chunk, int splits, int row_blocks,
                                                          int qt, int ot) {
    pdl_wait();
    pdl_trigger();                                            // after the wait: the join reads its inputs before its own
    using M = FewSmem<D, NT>;
    constexpr int R = 8 * NT, U = M::kStep, ST = M::kStages;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_rs[R], s_m[FEW_WARPS][R], s_l[FEW_WARPS][R], s_max[R], s_den[R], s_inv[R], s_lse[R];
    const int split = blockIdx.x % splits, rb = blockIdx.x / splits % row_blocks;
    const int sh = blockIdx.x / splits / row_blocks, head = sh % a.c.heads, s = sh / a.c.heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // Without a window this part starts at a place known before the sequence's length is: the page table entries of
    // the warp's first 32 tiles are read together with it (within the row of the table; used only if in the range).
    int early = -1;
    if (a.window == 0) {
        const int page = (split * (chunk / 16) + (warp + FEW_WARPS * (lane / U)) * U + lane % U) * 16 / a.c.page;
        if (page < a.sq.stride) early = a.sq.table[s * a.sq.stride + page];
    }
    const Seq q = load_seq(a.sq, s, a.c.page);
    const int n = min(q.n, a.max_tokens), r0 = rb * R, rows = min(n * a.group - r0, R);
    if (split == 0 && head == 0 && rb == 0 && threadIdx.x == 0) {
        const bool odd = a.sq.cu && odd_offsets(a.sq, s, a.sq.cu[s], a.sq.cu[s + 1]);
        if (odd || (rows > 0 && (q.n > n || min(q.end, a.max_kv) < q.len))) flag_error(DEVERR_LENGTH);
    }
    if (rows <= 0) return;
    const Range rg = visible_range(a, q, chunk);
    if (split >= rg.parts) return;
    const int first = q.len - q.n, end = min(q.end, a.max_kv);
    const int i0 = r0 / a.group, i1 = (r0 + rows - 1) / a.group;      // new tokens of the first and the last row
    // tiles of this part that some row of the block sees
    int t_begin = rg.tile0 + split * (chunk / 16), t_end = rg.tile0 + min(rg.tiles, (split + 1) * (chunk / 16));
    if (a.causal) t_end = min(t_end, (min(end, first + i1 + 1) + 15) / 16);
    if (a.window > 0) t_begin = max(t_begin, (first + i0 - a.window + 1) / 16);
    // this warp's steps of U tiles: the first at t_begin + U warp, the next 4U on; lane i looks up the place and the scales
    // of the i-th of the warp's next 32 tiles
    const int blocks = a.c.page / a.c.block;
    const int steps = max((t_end - t_begin - U * warp + U * FEW_WARPS - 1) / (U * FEW_WARPS), 0);
    long long src = 0;                                        // first code of the tile
    float ks = 0.f, lv = -INFINITY, iv = 0.f;                 // (no place: the tile's terms vanish)
    auto lookup = [&](int n0) {
        const int tile = t_begin + (warp + FEW_WARPS * ((n0 + lane) / U)) * U + (n0 + lane) % U, tok = tile * 16;
        src = 0, ks = 0.f, lv = -INFINITY, iv = 0.f;
        if (tile < t_end) {
            const int page = tok / a.c.page, off = tok - page * a.c.page;
            const int pg = n0 == 0 && a.window == 0 ? early : a.sq.table[s * a.sq.stride + page];
            if ((unsigned)pg < (unsigned long long)a.c.pages) {
                const int ph = pg * a.c.heads + head;
                src = ((long long)ph * a.c.page + off) * D;
                const long long sc = (long long)ph * blocks + off / a.c.block;
                ks = a.c.ks[sc];
                const float vs = fmaxf(a.c.vs[sc], SCALE_FLOOR);
                lv = __log2f(vs);
                iv = __fdividef(1.f, vs);
            } else {
                flag_error(DEVERR_PAGE);
            }
        }
    };
    float4* ring_scale = reinterpret_cast<float4*>(smem + M::kScale) + warp * (ST * U);
    uint8_t* ring = smem + M::kRing + warp * (ST * U * 2 * M::kTile);
    // copies of a step's tiles: lane -> chunk lane % (D/16) of rows lane / (D/16) + ...
    constexpr int CHUNKS = D / 16, PASS = 32 / CHUNKS;        // rows of one pass
    const int cr = lane / CHUNKS, cc = lane % CHUNKS;
    auto fetch = [&](int n) {
        if (n < steps) {
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int x = n * U + u, i = x & 31, slot = n % ST * U + u;
                if (i == 0 && x > 0) lookup(x);
                const long long at = __shfl_sync(0xffffffffu, src, i) + lane * 16;
                if (lane == i) ring_scale[slot] = make_float4(ks, lv, iv, 0.f);
                const uint32_t to = smem_u32(ring + slot * 2 * M::kTile);
#pragma unroll
                for (int r = 0; r < 16; r += PASS) {
                    cp_async_16(to + k_at<D>(r + cr, cc), a.c.k + at + r * D, 16);
                    cp_async_16(to + M::kTile + v_at<D>(r + cr, cc), a.c.v + at + r * D, 16);
                }
            }
        }
        cp_async_commit();
    };
    lookup(0);
#pragma unroll
    for (int n = 0; n < ST - 1; n++) fetch(n);               // on their way while the queries convert

    // queries to fp16, each row times the power of two that brings its largest magnitude to [1, 2)
    __half* sq = reinterpret_cast<__half*>(smem);
    constexpr int PER = D / 16;                               // values of a row for each of 16 lanes
    for (int r = threadIdx.x / 16; r < R; r += FEW_THREADS / 16) {
        const int l = threadIdx.x % 16;
        uint2 raw[PER / 4] = {};
        if (r < rows) {
            const uint2* p = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q.data) +
                                                            (long long)(q.n0 + (r0 + r) / a.group) * a.q.ts +
                                                            (long long)(head * a.group + (r0 + r) % a.group) * a.q.hs + l * PER);
#pragma unroll
            for (int i = 0; i < PER / 4; i++) raw[i] = p[i];
        }
        float x[PER], m = 0.f;
#pragma unroll
        for (int i = 0; i < PER / 4; i++) {
            Quad v;
            if (qt == MMQ_BF16) expand(raw[i], v, __nv_bfloat16());
            else expand(raw[i], v, __half());
            x[4 * i] = f2_lo(v[0]); x[4 * i + 1] = f2_hi(v[0]); x[4 * i + 2] = f2_lo(v[1]); x[4 * i + 3] = f2_hi(v[1]);
#pragma unroll
            for (int e = 0; e < 4; e++) m = fmaxf(m, fabsf(x[4 * i + e]));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float up, down;
        row_scale(m, up, down);
        uint2* to = reinterpret_cast<uint2*>(sq + r * (D + 8) + l * PER);
#pragma unroll
        for (int i = 0; i < PER / 4; i++)
            to[i] = make_uint2(pack2(x[4 * i] * up, x[4 * i + 1] * up, __half()),
                               pack2(x[4 * i + 2] * up, x[4 * i + 3] * up, __half()));
        if (l == 0) s_rs[r] = a.scale * LOG2E * down;
    }
    __syncthreads();
    // fragments of the queries: in registers, but for the largest shape, which reads them from shared memory each time
    constexpr bool QREG = D * NT <= 256;
    auto q_frag = [&](int nt, int w) {
        const uint2 v = *reinterpret_cast<const uint2*>(sq + (8 * nt + g) * (D + 8) + (w / 4) * 64 + 16 * t + 4 * (w % 4));
        return make_uint2(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632));
    };
    uint2 qf[QREG ? NT : 1][QREG ? D / 16 : 1];
    if constexpr (QREG) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int w = 0; w < D / 16; w++) qf[nt][w] = q_frag(nt, w);
    }
    float rs[NT][2], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            rs[nt][e] = s_rs[8 * nt + 2 * t + e];
            m[nt][e] = -INFINITY;
            l[nt][e] = 0.f;
        }
    // tiles whose 16 tokens every row sees need no mask
    const int lim_all = a.causal ? min(first + i0, end - 1) : end - 1;
    const int low_all = a.window > 0 ? first + i1 - a.window + 1 : 0;
    float o[D / 16][NT][4];
#pragma unroll
    for (int i = 0; i < D / 16; i++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[i][nt][e] = 0.f;

    for (int n = 0; n < steps; n++) {
        const int tok = (t_begin + (warp + FEW_WARPS * n) * U) * 16;
        cp_async_wait<ST - 2>();
        __syncwarp();                                         // every lane's copies of step n are here, step n-1 is read
        fetch(n + ST - 1);
        const uint32_t kv = smem_u32(ring + n % ST * U * 2 * M::kTile);
        const float4* scales = ring_scale + n % ST * U;
        float sc[U][NT][4], ivc[U];
        const bool masked = tok + 16 * U - 1 > lim_all || tok < low_all;
        bool grow = false;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t kt = kv + u * 2 * M::kTile;
            const float4 b = scales[u];
            ivc[u] = b.z;
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 4; e++) sc[u][nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 64; c++) {
                const uint4 ka = ld_shared_u4(kt + k_at<D>(g, 4 * c + t)), kb = ld_shared_u4(kt + k_at<D>(g + 8, 4 * c + t));
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    uint32_t a0, a1, a2, a3;
                    codes_even_odd(wa[w], a0, a2);
                    codes_even_odd(wb[w], a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        const uint2 f = QREG ? qf[QREG ? nt : 0][QREG ? 4 * c + w : 0] : q_frag(nt, 4 * c + w);
                        mma16816(sc[u][nt], a0, a1, a2, a3, f.x, f.y);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float f = rs[nt][e] * b.x;
                    sc[u][nt][e] = fmaf(sc[u][nt][e], f, b.y);
                    sc[u][nt][2 + e] = fmaf(sc[u][nt][2 + e], f, b.y);
                    if (masked) {
                        const int at = (r0 + min(8 * nt + 2 * t + e, rows - 1)) / a.group;   // new token of the row
                        const int lim = a.causal ? min(first + at, end - 1) : end - 1;
                        const int low = a.window > 0 ? first + at - a.window + 1 : 0, j = tok + 16 * u + g;
                        if (j > lim || j < low) sc[u][nt][e] = -INFINITY;
                        if (j + 8 > lim || j + 8 < low) sc[u][nt][2 + e] = -INFINITY;
                    }
                    grow |= fmaxf(sc[u][nt][e], sc[u][nt][2 + e]) > m[nt][e] + LAZY;
                }
        }
        // the reference of a row (one for the lanes that share its column) is raised when a term passes it by 2^LAZY
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float top = -INFINITY;
#pragma unroll
                    for (int u = 0; u < U; u++) top = fmaxf(top, fmaxf(sc[u][nt][e], sc[u][nt][2 + e]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    const float mn = fmaxf(m[nt][e], top - HEAD);
                    const float f = mn == -INFINITY ? 1.f : ex2(m[nt][e] - mn);
                    m[nt][e] = mn;
                    l[nt][e] *= f;
#pragma unroll
                    for (int d = 0; d < D / 16; d++) {
                        o[d][nt][e] *= f;
                        o[d][nt][2 + e] *= f;
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            uint32_t pf[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float mu = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
                    p[e] = ex2(sc[u][nt][e] - mu);
                    p[2 + e] = ex2(sc[u][nt][2 + e] - mu);
                    l[nt][e] = fmaf(p[e] + p[2 + e], ivc[u], l[nt][e]);
                }
                pf[nt][0] = transpose8(pack2(p[0], p[1], __half()));
                pf[nt][1] = transpose8(pack2(p[2], p[3], __half()));
            }
            // O^T += V^T P^T: a transposed read brings dimensions 2g, 2g+1 of 16-byte chunk c for tokens 2t, 2t+1 (and
            // + 8); fragment rows g, g+8 of product c are dimensions 16c + 2g and + 1
            const uint32_t vt = kv + (2 * u + 1) * M::kTile;
#pragma unroll
            for (int c = 0; c < D / 16; c += 2) {
                uint32_t vw[4];
                ldmatrix_trans(vt + v_at<D>(lane & 15, c + (lane >> 4)), vw);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    uint32_t a0, a1, a2, a3;
                    codes_even_odd(vw[2 * h], a0, a1);
                    codes_even_odd(vw[2 * h + 1], a2, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) mma16816(o[c + h][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                }
            }
        }
    }
    cp_async_wait<0>();

    // join the warps: common maximum, scaled sums through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            float x = l[nt][e];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            if (g == 0) {
                s_m[warp][8 * nt + 2 * t + e] = m[nt][e];
                s_l[warp][8 * nt + 2 * t + e] = x;
            }
        }
    __syncthreads();                                          // also: every warp has read its queries
    if (threadIdx.x < R) {
        const int r = threadIdx.x;
        float mx = s_m[0][r], den = 0.f;
#pragma unroll
        for (int w = 1; w < FEW_WARPS; w++) mx = fmaxf(mx, s_m[w][r]);
#pragma unroll
        for (int w = 0; w < FEW_WARPS; w++) den += s_l[w][r] * (s_m[w][r] == -INFINITY ? 0.f : ex2(s_m[w][r] - mx));
        s_max[r] = mx;
        s_den[r] = den;
        s_inv[r] = den == 0.f ? 0.f : 1.f / den;
        s_lse[r] = den == 0.f ? -INFINITY : LN2 * (mx + log2f(den));
    }
    float* so = reinterpret_cast<float*>(smem + FewSmem<D, NT>::kRing);
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int r = 8 * nt + 2 * t + e;
            float mx = s_m[0][r];
#pragma unroll
            for (int w = 1; w < FEW_WARPS; w++) mx = fmaxf(mx, s_m[w][r]);
            const float f = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - mx);
            float* row = so + (warp * R + r) * kSumPitch<D> + 2 * g;
#pragma unroll
            for (int c = 0; c < D / 16; c++)
                *reinterpret_cast<float2*>(row + 16 * c) = make_float2(o[c][nt][e] * f, o[c][nt][2 + e] * f);
        }
    __syncthreads();
    // four values of a row at a time; the rows' statistics by the first threads
    const long long all_rows = (long long)a.sq.tokens * a.heads;
    const bool whole = rg.parts == 1;
    for (int i = threadIdx.x; i < rows * (D / 4); i += FEW_THREADS) {
        const int r = i / (D / 4), d = 4 * (i % (D / 4));
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < FEW_WARPS; w++) {
            const float4 v = *reinterpret_cast<const float4*>(so + (w * R + r) * kSumPitch<D> + d);
            acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
        }
        const long long tok = q.n0 + (r0 + r) / a.group;
        const int h = head * a.group + (r0 + r) % a.group;
        if (whole) {
            const float f = s_inv[r];
#pragma unroll
            for (int e = 0; e < 4; e++) acc[e] = f == 0.f ? 0.f : acc[e] * f;
            store_out4(a.out.data, tok * a.out.ts + h * a.out.hs + d, acc, ot);
            if (d == 0 && a.lse) a.lse[tok * a.heads + h] = s_lse[r];
        } else {
            const long long row = split * all_rows + tok * a.heads + h;
            *reinterpret_cast<float4*>(a.part_o + row * D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (d == 0) a.part_ml[row] = make_float2(s_max[r], s_den[r]);
        }
    }
}

// Rows of split sequences: the parts' sums on a common maximum, in a fixed order.  W warps a row, each with
// eight parts' loads in flight: one where rows are many, four where they are fewer than resident blocks, eight for more
// parts than four warps take at once (131 k tokens 53.4 -> 52.7 us, 8 k tokens 11.0 -> 10.5; 8 parts 6.6 -> 6.8).
template <int W> constexpr int kJoinThreads = W == 8 ? 256 : 128;
template <int D, int W>
__global__ void __launch_bounds__(kJoinThreads<W>) join_kernel(const AttnArgs a, int chunk, int ot) {
    constexpr int ROWS = kJoinThreads<W> / 32 / W, PER = D / 32;
    __shared__ float s_acc[W > 1 ? W : 1][W > 1 ? D : 1], s_den[W];
    const long long all_rows = (long long)a.sq.tokens * a.heads;
    const long long row0 = (long long)blockIdx.x * ROWS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = W > 1 ? warp : 0;
    const long long row = W > 1 ? row0 : row0 + warp;
    const int t = (unsigned)min(row, all_rows - 1) / (unsigned)a.heads;
    // Lengths and offsets were complete before the attention kernel let this launch begin (its own wait comes first), so
    // they are read while that kernel still runs; its sums only after the wait below.
    int s = t;
    Seq q;
    if (a.sq.cu) {
        s = find_seq<kJoinThreads<W>>(a.sq, a.c.page, row0 / a.heads, [](int cu, int) { return (long long)cu; }, q);
        if (t >= q.n0 + q.n) {
            while (s + 1 < a.sq.seqs && a.sq.cu[s + 1] <= t) s++;
            q = load_seq(a.sq, s, a.c.page);
        }
    } else {
        q = load_seq(a.sq, s, a.c.page);
    }
    const bool mine = row < all_rows && t >= q.n0 && t < q.n0 + min(q.n, a.max_tokens);
    const int parts = visible_range(a, q, chunk).parts;
    pdl_wait();
    if (!mine || parts == 1) return;                          // W > 1: the whole block
    // the first eight parts before their weights are known
    float x[8][PER];
    auto fetch = [&](int p) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float* po = a.part_o + (min(p + W * i, parts - 1) * all_rows + row) * D + lane * PER;
            if constexpr (PER == 2) {
                const float2 v = *reinterpret_cast<const float2*>(po);
                x[i][0] = v.x; x[i][1] = v.y;
            } else {
#pragma unroll
                for (int e = 0; e < PER; e += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(po + e);
                    x[i][e] = v.x; x[i][e + 1] = v.y; x[i][e + 2] = v.z; x[i][e + 3] = v.w;
                }
            }
        }
    };
    fetch(w);
    float mx = -INFINITY;
    for (int p = lane; p < parts; p += 32) mx = fmaxf(mx, a.part_ml[p * all_rows + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float acc[PER], den = 0.f;
#pragma unroll
    for (int i = 0; i < PER; i++) acc[i] = 0.f;
    for (int p0 = w; p0 < parts; p0 += 32 * W) {              // lane i: weight of part p0 + W i
        const int its = p0 + W * lane;
        float f = 0.f;
        if (its < parts) {
            const float2 ml = a.part_ml[its * all_rows + row];
            f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx);
            den += ml.y * f;
        }
        const int here = min((parts - p0 + W - 1) / W, 32);
        for (int i0 = 0; i0 < here; i0 += 8) {
            if (p0 > w || i0 > 0) fetch(p0 + W * i0);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float fi = __shfl_sync(0xffffffffu, f, i0 + i);             // 0 past the last part
#pragma unroll
                for (int e = 0; e < PER; e++)                 // weight 0: past the last part, or nothing seen
                    acc[e] = fmaf(fi == 0.f ? 0.f : x[i][e], fi, acc[e]);
            }
        }
    }
    den = lane_sum<32>(den);
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < PER; e++) s_acc[w][lane * PER + e] = acc[e];
        if (lane == 0) s_den[w] = den;
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int u = 1; u < W; u++) {
            den += s_den[u];
#pragma unroll
            for (int e = 0; e < PER; e++) acc[e] += s_acc[u][lane * PER + e];
        }
    }
    const int h = (int)(row - (long long)t * a.heads);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const long long at = (long long)t * a.out.ts + h * a.out.hs + lane * PER;
    if constexpr (PER == 2) {
        const float x0 = inv == 0.f ? 0.f : acc[0] * inv, x1 = inv == 0.f ? 0.f : acc[1] * inv;
        if (ot == MMQ_F32) *reinterpret_cast<float2*>(static_cast<float*>(a.out.data) + at) = make_float2(x0, x1);
        else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out.data) + at) =
            ot == MMQ_BF16 ? pack2(x0, x1, __nv_bfloat16()) : pack2(x0, x1, __half());
    } else {
#pragma unroll
        for (int e = 0; e < PER; e += 4) {
            const float x[4] = {inv == 0.f ? 0.f : acc[e] * inv, inv == 0.f ? 0.f : acc[e + 1] * inv,
                                inv == 0.f ? 0.f : acc[e + 2] * inv, inv == 0.f ? 0.f : acc[e + 3] * inv};
            store_out4(a.out.data, at + e, x, ot);
        }
    }
    if (lane == 0 && a.lse) a.lse[row] = den == 0.f ? -INFINITY : LN2 * (mx + log2f(den));
}

template <int D, int NT>
cudaError_t launch_few(mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    const int row_blocks = (a.max_tokens * a.group + 8 * NT - 1) / (8 * NT);
    const long long grid = (long long)a.sq.seqs * a.c.heads * p.splits * row_blocks;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    constexpr int bytes = FewSmem<D, NT>::kBytes;
    auto kern = few_kernel<D, NT>;
    static bool configured[64] = {};
    bool& done = device_flag(configured);
    if (!done) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        done = true;
    }
    return launch_pdl_smem(kern, dim3((unsigned)grid), dim3(FEW_THREADS), bytes, s, a, p.chunk, p.splits, row_blocks,
                           (int)qt, (int)ot);
}

template <int D>
cudaError_t launch_few_rows(mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    return a.max_tokens * a.group <= 8 ? launch_few<D, 1>(qt, ot, a, p, s) : launch_few<D, 2>(qt, ot, a, p, s);
}

template <int D>
cudaError_t launch_join(int warps, long long grid, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    const dim3 g((unsigned)grid);
    if (warps == 8) return launch_pdl(join_kernel<D, 8>, g, dim3(kJoinThreads<8>), s, a, p.chunk, (int)ot);
    return launch_pdl(warps == 4 ? join_kernel<D, 4> : join_kernel<D, 1>, g, dim3(kJoinThreads<1>), s, a, p.chunk, (int)ot);
}

}  // namespace

cudaError_t run_attention_few(int dim, mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p,
                              cudaStream_t s) {
    switch (dim) {
        case 64: return launch_few_rows<64>(qt, ot, a, p, s);
        case 128: return launch_few_rows<128>(qt, ot, a, p, s);
        case 256: return launch_few_rows<256>(qt, ot, a, p, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t run_attention_join(int dim, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    const long long rows = (long long)a.sq.tokens * a.heads;
    const int warps = rows > 152 * 16 ? 1 : (p.splits > 32 ? 8 : 4);
    const long long grid = warps > 1 ? rows : (rows + 3) / 4;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    switch (dim) {
        case 64: return launch_join<64>(warps, grid, ot, a, p, s);
        case 128: return launch_join<128>(warps, grid, ot, a, p, s);
        case 256: return launch_join<256>(warps, grid, ot, a, p, s);
    }
    return cudaErrorInvalidValue;
}

MMQ_DEFINE_ERROR_READER(attn_few)

}  // namespace mmq
