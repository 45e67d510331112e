// attn_tiled.cu -- attention of many query rows (prompts, chunks of prompts) over the 8-bit paged cache, on tcgen05.
//
//   S = Q K^T (codes),  t_j = scale log2(e) ks_b S_j + log2(vs_b),  p_j = 2^(t_j - m),  O = sum_j p_j v_j (codes),
//   l = sum_b (1/vs_b) sum_{j in b} p_j,  out = O / l      (the same formulas as attn_few.cu)
//
// Bound by the tensor cores and the exponentials.  One thread block takes 256 rows (two tiles of 128; head_dim 256:
// one) of one sequence and key/value head, rows = (new token, query head of the group), and walks the cache in tiles
// of 128 tokens (head_dim 256: 64):
//   * four converter warps read the codes of a tile from their pages, turn them into fp16 exactly and store them
//     with the 128-byte swizzle.  K is the K-major operand of S, V the MN-major operand of O, so both have
//     the same layout [token][64 dimensions of 128 bytes] and one routine makes them.  Within each four dimensions
//     the order is 0 2 1 3 (two codes of a word convert at once); Q is stored in that order too, and the
//     output undoes it.  They also publish the tile's block scales.
//   * one warp issues the products, S_i = Q_i K^T into TMEM and O_i += P_i V with P_i from TMEM.  The two row
//     tiles alternate: while the softmax of one runs, the other's products do.
//   * four softmax warps for each row tile, one thread a row: two passes over the row of S in TMEM (maximum, then
//     exponentials), P as fp16 over the columns of S already read.  O is rescaled only when the maximum grows by
//     more than 2^8, which happens a few times in a row's life.
#include "attn_device.cuh"
#include "attn_math.cuh"
#include "internal.h"

namespace mmq {

namespace {

template <int D> struct Tiled {
    static constexpr int kQTiles = D == 256 ? 1 : 2;          // row tiles of 128
    static constexpr int kSBufs = 2;                          // S buffers: one a row tile, or two of one tile
    static constexpr int kTokens = D == 256 ? 64 : 128;       // cache tokens of a tile
    static constexpr int kStages = D == 64 ? 6 : 4;           // K and V tiles in turn
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kStageBytes = kTokens * D * 2;
    static constexpr int kBlocks = kTokens / 16;              // 16-token groups, each within a page and a scale block
    static constexpr int kScaleSlots = 4;
    // TMEM columns: S buffers (P over their first half), then O
    static constexpr int kOCol = kSBufs * kTokens;
    static constexpr int kCols = 512;
    static_assert(kOCol + kQTiles * D <= kCols, "TMEM budget");

    static constexpr int q_off = 0;
    static constexpr int kv_off = q_off + kQTiles * kQBytes;
    static constexpr int sc_off = kv_off + kStages * kStageBytes;              // float4 [slots][blocks]
    static constexpr int bar_off = sc_off + kScaleSlots * kBlocks * 16;
    static constexpr int n_bars = 2 * kStages + kScaleSlots + 3 * 2 + 1 + 2 + 1;
    static constexpr int misc_off = bar_off + n_bars * 8;
    static constexpr int alloc = misc_off + 16 + 1024;
    static_assert(alloc <= 232448, "shared memory budget");
};

constexpr int T_CONV0 = 8, T_CONV_WARPS = 4, T_MMA = 12;
constexpr int T_THREADS = 13 * 32;

// tcgen05.mma with A from TMEM (fp16, two elements a column).
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// MN-major operand with the 128-byte swizzle: 64 elements of MN contiguous, `slab` bytes to the next 64, 8-row groups
// of K 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t slab) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(slab >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

template <int D> struct TBars {
    using C = Tiled<D>;
    uint32_t b;
    __device__ uint32_t full(int i) const { return b + 8u * i; }                       // converters -> products
    __device__ uint32_t empty(int i) const { return b + 8u * (C::kStages + i); }
    __device__ uint32_t scale(int i) const { return b + 8u * (2 * C::kStages + i); }   // scales published
    __device__ uint32_t sfull(int i) const { return b + 8u * (2 * C::kStages + C::kScaleSlots + i); }
    __device__ uint32_t pready(int i) const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 2 + i); }
    __device__ uint32_t odone(int i) const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 4 + i); }
    __device__ uint32_t qfull() const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 6); }
    __device__ uint32_t pvdone() const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 7); }
    __device__ uint32_t done() const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 8); }
};

// The cache tiles [s, e) of a row tile, counted from the part's first token.
struct TileSpan {
    int s, e;
};

template <int D>
__global__ void __launch_bounds__(T_THREADS, 1) tiled_kernel(const AttnArgs a, int chunk, int splits, int q_blocks, int qt,
                                                             int ot) {
    using C = Tiled<D>;
    constexpr int KT = C::kTokens, NQ = C::kQTiles, ROWS = 128 * NQ;
    pdl_trigger();
    pdl_wait();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the last rows of a causal prompt see most of the cache: they go first
    const int per = a.sq.seqs * a.c.heads * splits;
    const int qb = q_blocks - 1 - (int)(blockIdx.x / per), rest = blockIdx.x % per;
    const int split = rest % splits, head = rest / splits % a.c.heads, s = rest / splits / a.c.heads;
    const Seq q = load_seq(a.sq, s, a.c.page);
    const int n = min(q.n, a.max_tokens), row0 = qb * ROWS, rows = min(n * a.group - row0, ROWS);
    if (rows <= 0) return;                                    // uniform, nothing set up yet
    if (split == 0 && head == 0 && qb == 0 && threadIdx.x == 0 && (q.n > n || min(q.end, a.max_kv) < q.len))
        flag_error(DEVERR_LENGTH);
    const Range rg = visible_range(a, q, chunk);
    if (split >= rg.parts) return;
    const int first = q.len - q.n, end = min(q.end, a.max_kv);
    const int base = (rg.tile0 + split * (chunk / 16)) * 16;                     // first token of this part
    const int stop = min(base + chunk, (rg.tile0 + rg.tiles) * 16);
    TileSpan span[NQ];
    int j0 = 1 << 30, j1 = 0;
#pragma unroll
    for (int i = 0; i < NQ; i++) {
        const int left = min(rows - 128 * i, 128);
        int lo = base, hi = min(stop, end);
        if (left > 0) {
            const int ta = first + (row0 + 128 * i) / a.group, tb = first + (row0 + 128 * i + left - 1) / a.group;
            if (a.causal) hi = min(hi, tb + 1);
            if (a.window > 0) lo = max(lo, ta - a.window + 1);
        } else {
            hi = lo;
        }
        span[i].s = (lo - base) / KT;
        span[i].e = hi > lo ? (hi - base + KT - 1) / KT : span[i].s;
        if (span[i].e > span[i].s) {
            j0 = min(j0, span[i].s);
            j1 = max(j1, span[i].e);
        }
    }
    if (j1 == 0) j0 = 0;                                      // no tile at all

    const uint32_t sb = smem_u32(smem);
    const TBars<D> bar{sb + C::bar_off};
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc_off + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc_off);
    float4* scales = reinterpret_cast<float4*>(smem + C::sc_off);
    if (warp == T_MMA) {
        if (lane == 0) {
            for (int i = 0; i < C::kStages; i++) {
                mbar_init(bar.full(i), T_CONV_WARPS);
                mbar_init(bar.empty(i), 1);
            }
            for (int i = 0; i < C::kScaleSlots; i++) mbar_init(bar.scale(i), T_CONV_WARPS);
            for (int i = 0; i < 2; i++) {
                mbar_init(bar.sfull(i), 1);
                mbar_init(bar.pready(i), 4);
                mbar_init(bar.odone(i), 1);
            }
            mbar_init(bar.qfull(), 4 * NQ);
            mbar_init(bar.pvdone(), 1);
            mbar_init(bar.done(), 1);
            *abort_flag = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), C::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp >= T_CONV0 && warp < T_CONV0 + T_CONV_WARPS) {
        // =========================================================== converters
        // warp w: rows w*KT/4 .. of the tile, in 16-token groups; lane (g, t): rows g, g+8 of a group, 16 bytes at
        // 16t of each 64.  A quarter-warp stores two rows of four 16-byte chunks: all 32 banks.
        constexpr int GROUPS = KT / 4 / 16, CH = D / 64;
        const int w = warp - T_CONV0, g = lane >> 2, t = lane & 3;
        const int blocks = a.c.page / a.c.block;
        int ph[GROUPS], off[GROUPS];                          // page and head, row in the page; ph < 0: zeros
        float ks = 0.f, lv = -INFINITY, iv = 0.f;             // lane i < GROUPS: scales of group i
        auto lookup = [&](int j) {
            int myph = -1, myoff = 0;
            ks = 0.f, lv = -INFINITY, iv = 0.f;
            if (lane < GROUPS && j < j1) {
                const int tok = base + j * KT + (w * GROUPS + lane) * 16;
                if (tok < end) {
                    const int page = tok / a.c.page;
                    myoff = tok - page * a.c.page;
                    const int pg = a.sq.table[s * a.sq.stride + page];
                    if ((unsigned)pg < (unsigned long long)a.c.pages) {
                        myph = pg * a.c.heads + head;
                        const long long sc = (long long)myph * blocks + myoff / a.c.block;
                        ks = a.c.ks[sc];
                        const float vs = fmaxf(a.c.vs[sc], SCALE_FLOOR);
                        lv = __log2f(vs);
                        iv = __fdividef(1.f, vs);
                    } else {
                        flag_error(DEVERR_PAGE);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < GROUPS; i++) {
                ph[i] = __shfl_sync(0xffffffffu, myph, i);
                off[i] = __shfl_sync(0xffffffffu, myoff, i);
            }
        };
        auto load = [&](const int8_t* codes, uint4 (&r)[GROUPS][2][CH]) {
#pragma unroll
            for (int i = 0; i < GROUPS; i++) {
                const int8_t* p = codes + ((long long)max(ph[i], 0) * a.c.page + off[i] + g) * D + 16 * t;
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int c = 0; c < CH; c++)
                        r[i][h][c] = ph[i] >= 0 ? ld_cache(p + 8 * h * D + 64 * c) : make_uint4(0, 0, 0, 0);
            }
        };
        auto store = [&](uint32_t tile, const uint4 (&r)[GROUPS][2][CH]) {
#pragma unroll
            for (int i = 0; i < GROUPS; i++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int row = (w * GROUPS + i) * 16 + 8 * h + g;
#pragma unroll
                    for (int c = 0; c < CH; c++) {
                        const uint4 x = r[i][h][c];
                        uint32_t y[8];
                        codes_even_odd(x.x, y[0], y[1]);
                        codes_even_odd(x.y, y[2], y[3]);
                        codes_even_odd(x.z, y[4], y[5]);
                        codes_even_odd(x.w, y[6], y[7]);
                        const uint32_t at = tile + c * KT * 128;
                        st_shared_v4(at + sw128_off(row, 2 * t), y[0], y[1], y[2], y[3]);
                        st_shared_v4(at + sw128_off(row, 2 * t + 1), y[4], y[5], y[6], y[7]);
                    }
                }
        };
        uint4 rk[GROUPS][2][CH], rv[GROUPS][2][CH];
        lookup(j0);
        load(a.c.k, rk);
        int it = 0;                                           // tiles stored, K and V
        for (int j = j0; j < j1; j++) {
            load(a.c.v, rv);
            // scales of this tile: the slot's last reader was four tiles ago (its S is complete)
            const int slot = (j - j0) % C::kScaleSlots;
            const float ks0 = ks, lv0 = lv, iv0 = iv;
            {
                const int st = it % C::kStages;
                if (!mbar_wait_relaxed(bar.empty(st), ((it / C::kStages) & 1) ^ 1, abort_flag)) break;
                if (lane < GROUPS) scales[slot * C::kBlocks + w * GROUPS + lane] = make_float4(ks0, lv0, iv0, 0.f);
                store(sb + C::kv_off + st * C::kStageBytes, rk);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar.full(st));
                    mbar_arrive(bar.scale(slot));
                }
                it++;
            }
            lookup(j + 1);
            if (j + 1 < j1) load(a.c.k, rk);
            {
                const int st = it % C::kStages;
                if (!mbar_wait_relaxed(bar.empty(st), ((it / C::kStages) & 1) ^ 1, abort_flag)) break;
                store(sb + C::kv_off + st * C::kStageBytes, rv);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.full(st));
                it++;
            }
        }
    } else if (warp == T_MMA) {
        // =========================================================== products
        constexpr uint32_t idesc_s = idesc_f16_f32(128, KT);
        constexpr uint32_t idesc_o = idesc_f16_f32(128, D) | (1u << 16);         // B is MN-major
        auto active = [&](int i, int j) { return j >= span[i].s && j < span[i].e; };
        auto product_s = [&](int i, int j) {                  // S of row tile i, cache tile j
            const int st = 2 * (j - j0) % C::kStages;
            const uint32_t qs = sb + C::q_off + i * C::kQBytes, kv = sb + C::kv_off + st * C::kStageBytes;
            const uint32_t buf = NQ == 2 ? i : (j - j0) & 1;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; k++)
                    umma_f16(tmem + buf * KT, sdesc_sw128(qs + (k / 4) * 16384) + 2 * (k % 4),
                             sdesc_sw128(kv + (k / 4) * KT * 128) + 2 * (k % 4), idesc_s, k > 0);
                umma_commit(bar.sfull(buf));
            }
            __syncwarp();
        };
        auto product_o = [&](int i, int j) {                  // O of row tile i
            const int st = (2 * (j - j0) + 1) % C::kStages;
            const uint32_t kv = sb + C::kv_off + st * C::kStageBytes;
            const uint32_t buf = NQ == 2 ? i : (j - j0) & 1;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < KT / 16; k++)
                    umma_f16_ts(tmem + C::kOCol + i * D, tmem + buf * KT + 8 * k,
                                sdesc_mn_sw128(kv + k * 2048, KT * 128), idesc_o, j > span[i].s || k > 0);
                if (j + 1 == span[i].e) umma_commit(bar.odone(i));
                if (NQ == 1) umma_commit(bar.pvdone());
            }
            __syncwarp();
        };
        auto wait_tile = [&](int x) {                         // x-th stored tile (K: even, V: odd)
            return mbar_wait(bar.full(x % C::kStages), (x / C::kStages) & 1, abort_flag);
        };
        auto release = [&](int x) {
            if (elect_one()) umma_commit(bar.empty(x % C::kStages));
            __syncwarp();
        };
        bool ok = j1 > j0 && mbar_wait(bar.qfull(), 0, abort_flag) && wait_tile(0);
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < NQ; i++)
                if (active(i, j0)) product_s(i, j0);
            release(0);
        }
        uint32_t np = 0;                                      // phase of each buffer's P
        for (int j = j0; ok && j < j1; j++) {
            const int x = 2 * (j - j0);
            const bool more = j + 1 < j1;
            if (NQ == 1 && more) {
                ok = wait_tile(x + 2);
                if (!ok) break;
                tc_fence_after();
                product_s(0, j + 1);
                release(x + 2);
            }
            ok = wait_tile(x + 1);
            if (!ok) break;
            if (NQ == 2 && more) ok = wait_tile(x + 2);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < NQ; i++) {
                if (active(i, j)) {
                    const int buf = NQ == 2 ? i : (j - j0) & 1;
                    ok = ok && mbar_wait(bar.pready(buf), (np >> buf) & 1, abort_flag);
                    np ^= 1u << buf;
                    if (!ok) break;
                    tc_fence_after();
                    product_o(i, j);
                }
                if (NQ == 2 && more && active(i, j + 1)) {
                    tc_fence_after();
                    product_s(i, j + 1);
                }
            }
            if (!ok) break;
            release(x + 1);
            if (NQ == 2 && more) release(x + 2);
        }
        if (elect_one()) umma_commit(bar.done());
        __syncwarp();
        mbar_wait_final(bar.done(), 0);
        __syncwarp();
    } else if (warp < 4 * NQ) {
        // =========================================================== softmax: one thread a row
        const int i = warp >> 2, r = 128 * i + (warp & 3) * 32 + lane;           // row of the block
        const bool real = r < rows;
        const int tokrow = (row0 + min(r, rows - 1)) / a.group;                   // new token
        const int hrow = head * a.group + (row0 + min(r, rows - 1)) % a.group;
        const long long tok = q.n0 + tokrow;
        float rs;
        {
            // the row to fp16, times the power of two that brings its largest magnitude to [1, 2); the sign of
            // the scale goes into the row
            const long long at = tok * a.q.ts + hrow * a.q.hs;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q.data) + at);
            float m = 0.f;
#pragma unroll 8
            for (int c = 0; c < D / 8; c++) {
                float x[8];
                unpack8(src[c], qt == MMQ_BF16, x);
#pragma unroll
                for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(x[e]));
            }
            float up, down;
            row_scale(m, up, down);
            if (!real) up = 0.f;
            if (a.scale < 0.f) up = -up;
            rs = fabsf(a.scale) * LOG2E * down;
#pragma unroll 8
            for (int c = 0; c < D / 8; c++) {
                float x[8];
                unpack8(src[c], qt == MMQ_BF16, x);
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 2; e++) {                 // dimension order 0 2 1 3
                    y[2 * e] = pack2(x[4 * e] * up, x[4 * e + 2] * up, __half());
                    y[2 * e + 1] = pack2(x[4 * e + 1] * up, x[4 * e + 3] * up, __half());
                }
                st_shared_v4(sb + C::q_off + i * C::kQBytes + (c / 8) * 16384 + sw128_off(r & 127, c % 8), y[0], y[1],
                             y[2], y[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.qfull());
        }
        const int lim = !real ? -1 : (a.causal ? min(first + tokrow, end - 1) : end - 1);
        const int low = a.window > 0 ? first + tokrow - a.window + 1 : 0;
        // tiles that every row of this warp sees whole need no mask
        const int ra = min(row0 + (r & ~31), row0 + rows - 1), rz = min(row0 + (r | 31), row0 + rows - 1);
        const int lim_all = a.causal ? min(first + ra / a.group, end - 1) : end - 1;
        const int low_all = a.window > 0 ? first + rz / a.group - a.window + 1 : 0;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t to = tmem + lanes + C::kOCol + i * D;
        float m = -INFINITY, l = 0.f;
        uint32_t ns = 0;                                      // phase of each buffer's S
        bool ok = true;
        for (int j = span[i].s; j < span[i].e; j++) {
            const int buf = NQ == 2 ? i : (j - j0) & 1, slot = (j - j0) % C::kScaleSlots;
            const uint32_t ts = tmem + lanes + buf * KT;
            if (!mbar_wait(bar.scale(slot), ((j - j0) / C::kScaleSlots) & 1, abort_flag) ||
                !mbar_wait(bar.sfull(buf), (ns >> buf) & 1, abort_flag)) {
                ok = false;
                break;
            }
            ns ^= 1u << buf;
            tc_fence_after();
            const float4* sc = scales + slot * C::kBlocks;
            const int t0 = base + j * KT;
            const bool masked = t0 + KT - 1 > lim_all || t0 < low_all;
            uint32_t va[32], vb[32];
            // pass 1: largest term of the row
            float top = -INFINITY;
            tmem_ld32(ts, va);
#pragma unroll
            for (int c = 0; c < KT / 32; c++) {
                uint32_t(&cur)[32] = (c & 1) ? vb : va;
                uint32_t(&nxt)[32] = (c & 1) ? va : vb;
                tmem_wait32(cur);
                tmem_ld32(ts + (c + 1 < KT / 32 ? 32 * (c + 1) : 0), nxt);        // the last one: pass 2's first
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float4 b = sc[2 * c + h];
                    const int tb = t0 + 32 * c + 16 * h;
                    float mx = -3.0e38f;
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 16; e++) {
                            const float x = __uint_as_float(cur[16 * h + e]);
                            mx = fmaxf(mx, (tb + e <= lim && tb + e >= low) ? x : -3.0e38f);
                        }
                        if (tb <= lim && tb + 15 >= low) top = fmaxf(top, fmaf(mx, b.x * rs, b.y));
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e++) mx = fmaxf(mx, __uint_as_float(cur[16 * h + e]));
                        top = fmaxf(top, fmaf(mx, b.x * rs, b.y));
                    }
                }
            }
            if (NQ == 1 && j > span[i].s) {                   // the product that reads and writes O is complete
                if (!mbar_wait(bar.pvdone(), (j - span[i].s - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
            }
            if (__any_sync(0xffffffffu, top > m + LAZY)) {
                const float mn = fmaxf(m, top);
                const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
                m = mn;
                l *= f;
                if (j > span[i].s) {                          // all products so far are complete: S came after them
                    tmem_wait32(va);
#pragma unroll 1
                    for (int c = 0; c < D / 16; c++) {
                        uint32_t o[16];
                        tmem_ld16(to + 16 * c, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int e = 0; e < 16; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st16(to + 16 * c, o);
                    }
                }
            }
            const float mu = m == -INFINITY ? 0.f : m;
            // pass 2: the terms, P over the columns of S that are read
#pragma unroll
            for (int c = 0; c < KT / 32; c++) {
                uint32_t(&cur)[32] = (c & 1) ? vb : va;
                uint32_t(&nxt)[32] = (c & 1) ? va : vb;
                tmem_wait32(cur);
                if (c + 1 < KT / 32) tmem_ld32(ts + 32 * (c + 1), nxt);
                uint32_t p[16];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float4 b = sc[2 * c + h];
                    const int tb = t0 + 32 * c + 16 * h;
                    const float f = b.x * rs, shift = b.y - mu;
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float p0 = ex2(fmaf(__uint_as_float(cur[16 * h + e]), f, shift));
                        float p1 = ex2(fmaf(__uint_as_float(cur[16 * h + e + 1]), f, shift));
                        if (masked) {
                            if (tb + e > lim || tb + e < low) p0 = 0.f;
                            if (tb + e + 1 > lim || tb + e + 1 < low) p1 = 0.f;
                        }
                        sum += p0 + p1;
                        p[8 * h + e / 2] = pack2(p0, p1, __half());
                    }
                    l = fmaf(sum, b.z, l);
                }
                tmem_st16(ts + 16 * c, p);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.pready(buf));
        }
        // ---- output row
        if (ok && span[i].e > span[i].s) {
            ok = mbar_wait(bar.odone(i), 0, abort_flag);
            tc_fence_after();
        }
        if (ok) {
            const bool none = span[i].e <= span[i].s;         // no tile: O was never written
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long all_rows = (long long)a.sq.tokens * a.heads, row = tok * a.heads + hrow;
            const bool part = rg.parts > 1;
            const float f = part ? 1.f : inv;
#pragma unroll 1
            for (int c = 0; c < D / 16; c++) {
                uint32_t o[16];
                if (!none) {
                    tmem_ld16(to + 16 * c, o);
                    tmem_ld_wait(o);
                }
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; e++) {                // column order 0 2 1 3 undone
                    const int d = (e & ~3) | ((e & 1) << 1) | ((e >> 1) & 1);
                    x[d] = none || f == 0.f ? 0.f : __uint_as_float(o[e]) * f;
                }
                if (real) {
                    if (part) store16(a.part_o + (split * all_rows + row) * D + 16 * c, x);
                    else store16_typed(a.out.data, tok * a.out.ts + hrow * a.out.hs + 16 * c, x, ot);
                }
            }
            if (real) {
                if (part) a.part_ml[split * all_rows + row] = make_float2(m, l);
                else if (a.lse) a.lse[row] = l == 0.f ? -INFINITY : LN2 * (m + log2f(l));
            }
        }
    }

    // ---- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == T_MMA) tmem_dealloc(tmem, C::kCols);
}

template <int D>
cudaError_t launch_tiled(mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    using C = Tiled<D>;
    const int q_blocks = (int)(((long long)a.max_tokens * a.group + 128 * C::kQTiles - 1) / (128 * C::kQTiles));
    const long long grid = (long long)a.sq.seqs * a.c.heads * p.splits * q_blocks;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    auto kern = tiled_kernel<D>;
    static bool configured[64] = {};
    bool& done = device_flag(configured);
    if (!done) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::alloc);
        if (e != cudaSuccess) return e;
        done = true;
    }
    return launch_pdl_smem(kern, dim3((unsigned)grid), dim3(T_THREADS), C::alloc, s, a, p.chunk, p.splits, q_blocks,
                           (int)qt, (int)ot);
}

}  // namespace

cudaError_t run_attention_tiled(int dim, mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p,
                                cudaStream_t s) {
    switch (dim) {
        case 64: return launch_tiled<64>(qt, ot, a, p, s);
        case 128: return launch_tiled<128>(qt, ot, a, p, s);
        case 256: return launch_tiled<256>(qt, ot, a, p, s);
    }
    return cudaErrorInvalidValue;
}

MMQ_DEFINE_ERROR_READER(attn_tiled)

}  // namespace mmq
