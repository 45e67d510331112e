// attn_tiled.cu -- attention of many query rows (prompts, chunks of prompts) over the 8-bit paged cache, on tcgen05.
//
//   S = Q K^T (codes),  t_j = scale log2(e) ks_b S_j + log2(vs_b),  p_j = 2^(t_j - m),  O = sum_j p_j v_j (codes),
//   l = sum_b (1/vs_b) sum_{j in b} p_j,  out = O / l      (the same formulas as attn_few.cu)
//
// Bound by the tensor cores and the exponentials.  One thread block takes 256 rows (two tiles of 128; head_dim 256:
// one) of one sequence and key/value head, rows = (new token, query head of the group), and walks the cache in tiles
// of 128 tokens (head_dim 256: 64):
//   * seven converter warps read the codes in units of 32 tokens (two groups of 16, each within one page), turn them into
//     fp16 exactly and store them with the 128-byte swizzle.  K is the K-major operand of S, V the MN-major operand of
//     O, so both have the same layout [token][64 dimensions of 128 bytes] and one routine makes them.  Within each
//     four dimensions the order is 0 2 1 3 (two codes of a word convert at once); Q is stored in that order too, and
//     the output undoes it.  They also publish the groups' block scales.
//   * one warp issues the products, S_i = Q_i K^T into TMEM and O_i += P_i V with P_i from TMEM.  The two row
//     tiles alternate: while the softmax of one runs, the other's products do.
//   * four softmax warps for each row tile, one thread a row: the row of S in registers, its maximum, the
//     exponentials, P as fp16 over the columns of S (in halves, so that the product can start on the first).  O is
//     rescaled only when the maximum outgrows its slack (LAZY), which happens a few times in a row's life.  These warps
//     also bring the queries in and the outputs out, as whole rows through shared memory.
// What it measures (GB300; 1909 TFLOP/s is the card's dense fp16 rate): 2048 tokens of 16 heads after 30000 cached ones,
// 389 us, 1.34 PFLOP/s; prompts of up to 4096 tokens of 32 heads, 308 us, 1.03 PFLOP/s.  A tile of 128 tokens takes a
// block 3300 cycles: 1700 to 2000 of products (their operands take 1500 cycles of shared memory reads, the converted
// codes 500 of writes), the rest is the chain S -> maximum -> exponentials -> P, which two row tiles hide in part.
// Variants measured slower: two threads a row (chunk 492 -> 625 us), the reference checked after the exponentials
// instead of a maximum first (492 -> 525), each half of P on its own maximum (394 -> 413), P in one piece (394 -> 399),
// three or six converter warps (691, 413), parts and rests of equal length, S in halves of 64 tokens with the first made
// ahead over columns already read (393 -> 483: the queries are read from shared memory twice).
#include "attn_device.cuh"
#include "attn_math.cuh"
#include "internal.h"

namespace mmq {

namespace {

template <int D> struct Tiled {
    static constexpr int kQTiles = D == 256 ? 1 : 2;          // row tiles of 128
    static constexpr int kSBufs = 2;                          // S buffers: one a row tile, or two of one tile
    static constexpr int kTokens = D == 256 ? 64 : 128;       // cache tokens of a tile
    static constexpr int kStages = D == 64 ? 6 : 5;           // K and V tiles in turn
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kStageBytes = kTokens * D * 2;
    static constexpr int kBlocks = kTokens / 16;              // 16-token groups, each within a page and a scale block
    static constexpr int kScaleSlots = 4;
    // registers a thread, moved from the converter and product warps to the softmax warps (a row of S each)
    static constexpr int kRegsSoftmax = D == 256 ? 128 : 176, kRegsRest = D == 256 ? 128 : 80;
    static_assert(kRegsSoftmax + kRegsRest <= 256, "register budget: as many warps of either kind, 128 at launch");
    // TMEM columns: S buffers (P over their first half), then O
    static constexpr int kOCol = kSBufs * kTokens;
    static constexpr int kCols = 512;
    static_assert(kOCol + kQTiles * D <= kCols, "TMEM budget");

    static constexpr int q_off = 0;
    static constexpr int kv_off = q_off + kQTiles * kQBytes;
    static constexpr int sc_off = kv_off + kStages * kStageBytes;              // float4 [slots][blocks]
    static constexpr int bar_off = sc_off + kScaleSlots * kBlocks * 16;
    static constexpr int n_bars = 2 * kStages + kScaleSlots + 2 + 4 + 2 + 3;
    static constexpr int misc_off = bar_off + n_bars * 8;
    static constexpr int alloc = misc_off + 16 + 1024;
    static_assert(alloc <= 232448, "shared memory budget");
};

constexpr int T_CONV0 = 8, T_CONV_WARPS = 7, T_MMA = 15;
constexpr int T_THREADS = 16 * 32;
constexpr float MASKED = -3.0e38f;           // a hidden score: its term is below NOTHING for any scale above F_FLOOR
constexpr float F_FLOOR = 1e-30f;
constexpr float NOTHING = -1e8f;

// Shared-memory matrix descriptors as two words: the upper one is constant for a layout (8-row groups 1024 bytes
// apart, 128-byte swizzle), the lower one holds the start address / 16 and the leading offset / 16, so that stepping
// along an operand adds to the lower word.  K-major: leading offset unused (1).  MN-major (64 elements of MN contiguous):
// leading offset = bytes to the next 64 elements of MN.
constexpr uint32_t DESC_HI = (uint32_t)(((uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61) >> 32);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading) {
    return ((saddr & 0x3FFFFu) >> 4) | (leading >> 4) << 16;
}
// D[tmem] (+)= A[smem] B[smem]^T, and with A from TMEM (fp16, two elements a column).
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(DESC_HI)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "r"(DESC_HI)
        : "memory");
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
// 64 columns of 32-bit TMEM values for this warp's 32 lanes, and the wait that makes them usable.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait64(uint32_t (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]),
                   "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]),
                   "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]),
                   "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]),
                   "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
                 :
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <int D> struct TBars {
    using C = Tiled<D>;
    uint32_t b;
    __device__ uint32_t full(int i) const { return b + 8u * i; }                       // converters -> products
    __device__ uint32_t empty(int i) const { return b + 8u * (C::kStages + i); }
    __device__ uint32_t scale(int i) const { return b + 8u * (2 * C::kStages + i); }   // scales published
    __device__ uint32_t sfull(int i) const { return b + 8u * (2 * C::kStages + C::kScaleSlots + i); }
    __device__ uint32_t pready(int i, int h) const {                                   // halves of P
        return b + 8u * (2 * C::kStages + C::kScaleSlots + 2 + 2 * i + h);
    }
    __device__ uint32_t odone(int i) const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 6 + i); }
    __device__ uint32_t qfull() const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 8); }
    __device__ uint32_t pvdone() const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 9); }
    __device__ uint32_t done() const { return b + 8u * (2 * C::kStages + C::kScaleSlots + 10); }
};

// The cache tiles [s, e) of a row tile, counted from the part's first token.
struct TileSpan {
    int s, e;
};

// PACKED: row blocks numbered through the packed rows instead of for every sequence the most that one has.
// LONG: parts may be longer than kChain tokens, after which the sums are put aside.
template <int D, bool PACKED, bool LONG>
__global__ void __launch_bounds__(T_THREADS, 1) tiled_kernel(const AttnArgs a, int chunk, int slots, int qt, int ot) {
    using C = Tiled<D>;
    constexpr int KT = C::kTokens, NQ = C::kQTiles, ROWS = 128 * NQ;
    pdl_wait();
    pdl_trigger();                                            // after the wait: the join reads its inputs before its own
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // Long pieces first: a range's whole parts before its last one, and the last rows, which see most of a causal prompt's
    // cache, before the others.
    Seq q;
    int s, qb, head, split;
    if constexpr (PACKED) {                                   // block cu[s]*group/ROWS + s is the first of sequence s
        const int piece = blockIdx.x / a.c.heads, slot = slots - 1 - piece % slots;
        head = blockIdx.x % a.c.heads;
        split = piece / slots;
        auto first_block = [&](int cu, int i) { return (long long)cu * a.group / ROWS + i; };
        s = find_seq<T_THREADS>(a.sq, a.c.page, slot, first_block, q);
        qb = slot - (int)first_block(q.n0, s);
    } else {
        const int per = a.sq.seqs * a.c.heads, piece = blockIdx.x / per, sh = blockIdx.x % per;
        split = piece / slots;
        qb = slots - 1 - piece % slots;
        head = sh % a.c.heads;
        s = sh / a.c.heads;
        q = load_seq(a.sq, s, a.c.page);
        if (split == 0 && head == 0 && qb == 0 && threadIdx.x == 0 && a.sq.cu &&
            odd_offsets(a.sq, s, a.sq.cu[s], a.sq.cu[s + 1]))
            flag_error(DEVERR_LENGTH);
    }
    const int n = min(q.n, a.max_tokens), row0 = qb * ROWS, rows = min(n * a.group - row0, ROWS);
    if (rows <= 0 || qb < 0) return;                          // uniform, nothing set up yet
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
    // The softmax warps' rows of queries come whole by asynchronous copies, D/8 lanes on a row, to where the operand
    // belongs, while the block is set up (prompts: 309 us with the copies after it, 303).
    constexpr int LPR = D / 8, RPS = 32 / LPR;                // lanes on a row, rows at a time
    const int sub = lane % LPR;
    if (warp < 4 * NQ) {
        const int r = min(warp * 32 + lane, rows - 1);
        const long long mine = ((long long)(q.n0 + (row0 + r) / a.group) * a.q.ts +
                                (long long)(head * a.group + (row0 + r) % a.group) * a.q.hs) * 2;
        const uint8_t* src = static_cast<const uint8_t*>(a.q.data) + sub * 16;
        const uint32_t tile = sb + C::q_off + (warp >> 2) * C::kQBytes;
#pragma unroll 8
        for (int s0 = 0; s0 < 32; s0 += RPS) {
            const int at = s0 + lane / LPR;                   // row of the warp
            cp_async_16(tile + (sub / 8) * 16384 + sw128_off((warp & 3) * 32 + at, sub % 8),
                        src + __shfl_sync(0xffffffffu, mine, at), 16);
        }
        cp_async_commit();
    }
    if (warp == T_MMA) {
        if (lane == 0) {
            for (int i = 0; i < C::kStages; i++) {
                mbar_init(bar.full(i), KT / 32);
                mbar_init(bar.empty(i), 1);
            }
            for (int i = 0; i < C::kScaleSlots; i++) mbar_init(bar.scale(i), KT / 32);
            for (int i = 0; i < 2; i++) {
                mbar_init(bar.sfull(i), 1);
                mbar_init(bar.pready(i, 0), 4);
                mbar_init(bar.pready(i, 1), 4);
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
    // The roles stand inside the branch that sets their share of registers (not indented further): set in a branch before
    // theirs, the compiler keeps to the launch's 128 and spills 4 KB a thread.
    if (warp >= T_CONV0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    if (warp != T_MMA) {
        // =========================================================== converters
        // Units of 32 tokens (two groups of 16, each within one page), K's of a tile and then V's; warp w takes every
        // seventh.  Lane (g, t) of a group: rows g, g+8, 16 bytes at 16t of each 64.  A quarter-warp stores two rows
        // of four 16-byte chunks: all 32 banks.
        constexpr int CH = D / 64, UNITS = KT / 32;           // units of a stored tile
        const int w = warp - T_CONV0, g = lane >> 2, t = lane & 3;
        const int blocks = a.c.page / a.c.block, units = (j1 - j0) * 2 * UNITS;
        const uint32_t sts0 = sb + C::kv_off + sw128_off(g, 2 * t), sts1 = sb + C::kv_off + sw128_off(g, 2 * t + 1);
        // lanes 2i, 2i+1 look up the groups of the i-th of the warp's next 16 units
        long long src = -1;                                   // first code of the group (negative: zeros)
        float ks = 0.f, lv = -INFINITY, iv = 0.f;
        auto lookup = [&](int u0) {
            const int u = u0 + T_CONV_WARPS * (lane >> 1);
            src = -1, ks = 0.f, lv = -INFINITY, iv = 0.f;
            const int tok = base + (j0 + u / (2 * UNITS)) * KT + (u % UNITS) * 32 + (lane & 1) * 16;
            if (u < units && tok < end) {
                const int page = tok / a.c.page, off = tok - page * a.c.page;
                const int pg = a.sq.table[s * a.sq.stride + page];
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
        uint4 r[2][2][CH];
        auto load = [&](int x, int i) {                       // i-th looked-up unit, of stored tile x
            const int8_t* codes = (x & 1 ? a.c.v : a.c.k) + g * D + 16 * t;
#pragma unroll
            for (int q2 = 0; q2 < 2; q2++) {
                const long long at = __shfl_sync(0xffffffffu, src, 2 * i + q2);
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int c = 0; c < CH; c++)
                        r[q2][h][c] = at >= 0 ? ld_cache(codes + at + 8 * h * D + 64 * c) : make_uint4(0, 0, 0, 0);
            }
        };
        // A barrier shows a phase's parity only, so a warp must not be two phases off.  It is not lapped, since its
        // own unit completes the tile; and as stages are released in the order of the tiles, the wait for its unit
        // before, at most kStages tiles back, shows that the phase before this one is complete.
        static_assert((T_CONV_WARPS + UNITS - 1) / UNITS <= C::kStages, "a warp's units at most kStages tiles apart");
        int i = 0;
        lookup(w);
        if (w < units) load(w / UNITS, 0);
        for (int u = w; u < units; u += T_CONV_WARPS) {
            const int x = u / UNITS, st = x % C::kStages, unit = u % UNITS;      // stored tile x
            if (!mbar_wait(bar.empty(st), ((x / C::kStages) & 1) ^ 1, abort_flag)) break;
            const uint32_t to = st * C::kStageBytes + unit * 32 * 128;
#pragma unroll
            for (int q2 = 0; q2 < 2; q2++)
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int c = 0; c < CH; c++) {
                        const uint4 v = r[q2][h][c];
                        uint32_t y[8];
                        codes_even_odd(v.x, y[0], y[1]);
                        codes_even_odd(v.y, y[2], y[3]);
                        codes_even_odd(v.z, y[4], y[5]);
                        codes_even_odd(v.w, y[6], y[7]);
                        const uint32_t at = to + c * KT * 128 + q2 * 2048 + h * 1024;
                        st_shared_v4(sts0 + at, y[0], y[1], y[2], y[3]);
                        st_shared_v4(sts1 + at, y[4], y[5], y[6], y[7]);
                    }
            // scales with the K units; the slot's last reader was four tiles ago (its S is complete)
            const int slot = (x >> 1) % C::kScaleSlots;
            if (!(x & 1) && (lane >> 1) == i) scales[slot * C::kBlocks + 2 * unit + (lane & 1)] = make_float4(ks, lv, iv, 0.f);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar.full(st));
                if (!(x & 1)) mbar_arrive(bar.scale(slot));
            }
            if (++i == 16) {
                lookup(u + T_CONV_WARPS);
                i = 0;
            }
            if (u + T_CONV_WARPS < units) load((u + T_CONV_WARPS) / UNITS, i);
        }
    } else {
        // =========================================================== products
        constexpr uint32_t idesc_s = idesc_f16_f32(128, KT);
        constexpr uint32_t idesc_o = idesc_f16_f32(128, D) | (1u << 16);         // B is MN-major
        const uint32_t q_lo = desc_lo(sb + C::q_off, 16), k_lo = desc_lo(sb + C::kv_off, 16);
        const uint32_t v_lo = desc_lo(sb + C::kv_off, KT * 128);
        auto active = [&](int i, int j) { return j >= span[i].s && j < span[i].e; };
        auto product_s = [&](int i, int j) {                  // S of row tile i, cache tile j
            const int st = 2 * (j - j0) % C::kStages;
            const uint32_t qs = q_lo + i * (C::kQBytes >> 4), kv = k_lo + st * (C::kStageBytes >> 4);
            const uint32_t buf = NQ == 2 ? i : (j - j0) & 1;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; k++)
                    umma_ss(tmem + buf * KT, qs + (k / 4) * (16384 >> 4) + 2 * (k % 4),
                            kv + (k / 4) * (KT * 128 >> 4) + 2 * (k % 4), idesc_s, k > 0);
                umma_commit(bar.sfull(buf));
            }
            __syncwarp();
        };
        auto product_o = [&](int i, int j, int h) {           // O of row tile i, half h of the cache tile's tokens
            const int st = (2 * (j - j0) + 1) % C::kStages;
            const uint32_t kv = v_lo + st * (C::kStageBytes >> 4);
            const uint32_t buf = NQ == 2 ? i : (j - j0) & 1;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < KT / 32; k++) {
                    const int kk = h * (KT / 32) + k;
                    umma_ts(tmem + C::kOCol + i * D, tmem + buf * KT + 8 * kk, kv + kk * (2048 >> 4), idesc_o,
                            j > span[i].s || kk > 0);
                }
                if (h == 1 && j + 1 == span[i].e) umma_commit(bar.odone(i));
                if (h == 1 && NQ == 1) umma_commit(bar.pvdone());
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
            }
            ok = wait_tile(x + 1);
            if (!ok) break;
            if (NQ == 2 && more) ok = wait_tile(x + 2);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < NQ; i++) {
                if (active(i, j)) {
                    const int buf = NQ == 2 ? i : (j - j0) & 1;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        ok = ok && mbar_wait(bar.pready(buf, h), (np >> buf) & 1, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        product_o(i, j, h);
                    }
                    np ^= 1u << buf;
                    if (!ok) break;
                }
                if (i == NQ - 1) release(x + 1);
                if (NQ == 2 && more && active(i, j + 1)) {
                    tc_fence_after();
                    product_s(i, j + 1);
                }
            }
            if (!ok) break;
            if (more) release(x + 2);
        }
        if (elect_one()) umma_commit(bar.done());
        __syncwarp();
        mbar_wait_final(bar.done(), 0);
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    if (warp < 4 * NQ) {
        // =========================================================== softmax: one thread a row
        const int i = warp >> 2, r = 128 * i + (warp & 3) * 32 + lane;           // row of the block
        const bool real = r < rows;
        const int tokrow = (row0 + min(r, rows - 1)) / a.group;                   // new token
        const int hrow = head * a.group + (row0 + min(r, rows - 1)) % a.group;
        const long long tok = q.n0 + tokrow;
        float rs = 0.f;
        {
            // Each thread turns its row into fp16 in place, times the power of two that brings the row's largest
            // magnitude to [1, 2) (the sign of the scale goes into the row).
            const uint32_t tile = sb + C::q_off + i * C::kQBytes;
            cp_async_wait<0>();
            __syncwarp();
            // magnitudes order as the integers that their bits are, in both 16-bit types
            unsigned big[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
            for (int c = 0; c < D / 8; c++) {
                const uint4 v = ld_shared_u4(tile + (c / 8) * 16384 + sw128_off(r & 127, c % 8));
                big[0] = __vmaxu2(big[0], v.x & 0x7FFF7FFFu);
                big[1] = __vmaxu2(big[1], v.y & 0x7FFF7FFFu);
                big[2] = __vmaxu2(big[2], v.z & 0x7FFF7FFFu);
                big[3] = __vmaxu2(big[3], v.w & 0x7FFF7FFFu);
            }
            const unsigned pair = __vmaxu2(__vmaxu2(big[0], big[1]), __vmaxu2(big[2], big[3]));
            const unsigned short top = (unsigned short)max(pair & 0xFFFFu, pair >> 16);
            const float m = qt == MMQ_BF16 ? __uint_as_float((unsigned)top << 16) : half_bits_to_float(top);
            float up, down;
            row_scale(m, up, down);
            if (!real) up = 0.f;
            if (a.scale < 0.f) up = -up;
            rs = fabsf(a.scale) * LOG2E * down;
#pragma unroll 4
            for (int c = 0; c < D / 8; c++) {
                const uint32_t place = tile + (c / 8) * 16384 + sw128_off(r & 127, c % 8);
                float x[8];
                unpack8(ld_shared_u4(place), qt == MMQ_BF16, x);
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 2; e++) {                 // dimension order 0 2 1 3
                    y[2 * e] = pack2(x[4 * e] * up, x[4 * e + 2] * up, __half());
                    y[2 * e + 1] = pack2(x[4 * e + 1] * up, x[4 * e + 3] * up, __half());
                }
                st_shared_v4(place, y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.qfull());
        }
        // in the loop everything counts from the first tile: tiles kt, columns that the row sees, and the tiles that every
        // row of this warp sees whole and that need no mask
        const int b0 = base + j0 * KT, k_s = span[i].s - j0, k_e = span[i].e - j0;
        const int lim = (!real ? -1 : (a.causal ? min(first + tokrow, end - 1) : end - 1)) - b0;
        const int low = (a.window > 0 ? first + tokrow - a.window + 1 : 0) - b0;
        const int ra = min(row0 + (r & ~31), row0 + rows - 1), rz = min(row0 + (r | 31), row0 + rows - 1);
        const int k_hi = max((a.causal ? min(first + ra / a.group, end - 1) : end - 1) - b0 + 1, 0) / KT;
        const int k_lo = a.window > 0 ? (max(first + rz / a.group - a.window + 1 - b0, 0) + KT - 1) / KT : 0;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t to = tmem + lanes + C::kOCol + i * D;
        // Tiles summed in one go, and the row's place for such sums (worked out where it is needed: the rows are hidden from
        // the compiler, which would keep it in registers throughout).
        constexpr int CHAIN = kChain / KT;
        auto place = [&]() {
            int at = min(r, rows - 1);
            asm volatile("" : "+r"(at));
            return (long long)split * a.sq.tokens * a.heads + (q.n0 + (row0 + at) / a.group) * (long long)a.heads +
                   head * a.group + (row0 + at) % a.group;
        };
        float m = -INFINITY, l = 0.f, lost = 0.f;
        uint32_t ns = 0;                                      // phase of each buffer's S
        bool ok = true;
        for (int k = k_s; k < k_e; k++) {
            const int buf = NQ == 2 ? i : k & 1, slot = k % C::kScaleSlots;
            const uint32_t ts = tmem + lanes + buf * KT;
            if (!mbar_wait(bar.scale(slot), (k / C::kScaleSlots) & 1, abort_flag) ||
                !mbar_wait(bar.sfull(buf), (ns >> buf) & 1, abort_flag)) {
                ok = false;
                break;
            }
            ns ^= 1u << buf;
            tc_fence_after();
            if (LONG && k % CHAIN == 0 && k > k_s) {
                // The accumulators are truncated after every 16 tokens, always to the same side: by up to 2^-22 of what they
                // hold, 2^-9 after 131 k tokens.  So every kChain tokens O goes to the row's place in the workspace, with
                // its l and reference, and starts from zero.  All products so far are complete: S came after them (or the
                // last one is waited for).
                if (NQ == 1) {
                    if (!mbar_wait(bar.pvdone(), (k - k_s - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                const long long at = place();
                float2 was = make_float2(-INFINITY, 0.f);
                if (real && k - CHAIN > k_s) was = a.part_ml[at];
                const float f = was.x == -INFINITY ? 0.f : ex2(was.x - m);
#pragma unroll 1
                for (int c = 0; c < D / 16; c++) {
                    uint32_t o[16];
                    tmem_ld16(to + 16 * c, o);
                    tmem_ld_wait(o);
                    if (real) {
                        float4* aside = reinterpret_cast<float4*>(a.part_o + at * D + 16 * c);
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (f != 0.f) v = aside[e];
                            aside[e] = make_float4(fmaf(v.x, f, __uint_as_float(o[4 * e])),
                                                   fmaf(v.y, f, __uint_as_float(o[4 * e + 1])),
                                                   fmaf(v.z, f, __uint_as_float(o[4 * e + 2])),
                                                   fmaf(v.w, f, __uint_as_float(o[4 * e + 3])));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; e++) o[e] = 0u;
                    tmem_st16(to + 16 * c, o);
                }
                if (real) a.part_ml[at] = make_float2(m, fmaf(was.y, f, l));
                l = lost = 0.f;
            }
            const float4* sc = scales + slot * C::kBlocks;
            const bool masked = k < k_lo || k >= k_hi;
            float x[KT];                                      // the row of S
            {
                uint32_t(&v)[KT / 64][64] = reinterpret_cast<uint32_t(&)[KT / 64][64]>(x);
#pragma unroll
                for (int c = 0; c < KT / 64; c++) tmem_ld64(ts + 64 * c, v[c]);
#pragma unroll
                for (int c = 0; c < KT / 64; c++) tmem_wait64(v[c]);
            }
            if (masked) {
                const int hi = lim - k * KT, lo = low - k * KT;
#pragma unroll
                for (int e = 0; e < KT; e++)
                    if (e > hi || e < lo) x[e] = MASKED;
            }
            float top = -INFINITY;
#pragma unroll
            for (int g = 0; g < KT / 16; g++) {
                const float* v = x + 16 * g;
                float m0 = max3(v[0], v[1], v[2]), m1 = max3(v[3], v[4], v[5]), m2 = max3(v[6], v[7], v[8]);
                m0 = max3(m0, v[9], v[10]);
                m1 = max3(m1, v[11], v[12]);
                m2 = max3(m2, v[13], v[14]);
                m0 = fmaxf(max3(m0, m1, m2), v[15]);
                const float4 b = sc[g];
                top = fmaxf(top, fmaf(m0, fmaxf(b.x * rs, F_FLOOR), b.y));
            }
            if (top < NOTHING) top = -INFINITY;
            if (NQ == 1 && k > k_s) {                   // the product that reads and writes O is complete
                if (!mbar_wait(bar.pvdone(), (k - k_s - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
            }
            if (__any_sync(0xffffffffu, top > m + LAZY)) {
                const float mn = fmaxf(m, top - HEAD);
                const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
                m = mn;
                l *= f;
                lost *= f;
                if (k > k_s) {                                // all products so far are complete: S came after them
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
            float add = 0.f;
#pragma unroll
            for (int h = 0; h < 2; h++) {
#pragma unroll
                for (int c = 0; c < KT / 64; c++) {           // 32 columns: two blocks
                    uint32_t p[16];
#pragma unroll
                    for (int k2 = 0; k2 < 2; k2++) {
                        const int g = h * (KT / 32) + 2 * c + k2;
                        const float4 b = sc[g];
                        const float f = fmaxf(b.x * rs, F_FLOOR), shift = b.y - mu;
                        const uint64_t f2 = f2_pack(f, f), s2 = f2_pack(shift, shift);
                        uint64_t sum2 = 0ull;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float p0, p1;
                            f2_unpack(f2_fma(f2_pack(x[16 * g + e], x[16 * g + e + 1]), f2, s2), p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            sum2 = f2_add(sum2, f2_pack(p0, p1));
                            p[8 * k2 + e / 2] = pack2(p0, p1, __half());
                        }
                        float a0, a1;
                        f2_unpack(sum2, a0, a1);
                        add = fmaf(a0 + a1, b.z, add);
                    }
                    tmem_st16(ts + (h * (KT / 64) + c) * 16, p);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.pready(buf, h));
            }
            // One rounding a tile: 2^-24 of l to the same side, at most 256 times before l is put aside (with one for every 16 tokens, lse
            // was off by 4e-4 after 131 k tokens); the shorter tiles of head_dim 256 carry on what was rounded away.  All of
            // them doing so costs 0.5 %.
            if constexpr (KT < 128) {
                const float y = add - lost, sum = l + y;
                lost = (sum - l) - y;
                l = sum;
            } else {
                l += add;
            }
        }
        // ---- output row
        if (ok && span[i].e > span[i].s) {
            ok = mbar_wait(bar.odone(i), 0, abort_flag);
            tc_fence_after();
        }
        if (LONG && ok && (k_e - 1) / CHAIN * CHAIN > k_s) {  // what was put aside, on the last reference
            const long long at = place();
            float2 was = make_float2(-INFINITY, 0.f);
            if (real) was = a.part_ml[at];
            const float f = was.x == -INFINITY ? 0.f : ex2(was.x - m);
            l = fmaf(was.y, f, l);
#pragma unroll 1
            for (int c = 0; c < D / 16; c++) {
                uint32_t o[16];
                tmem_ld16(to + 16 * c, o);
                tmem_ld_wait(o);
                if (f != 0.f) {
                    const float* aside = a.part_o + at * D + 16 * c;
#pragma unroll
                    for (int e = 0; e < 16; e++) o[e] = __float_as_uint(fmaf(aside[e], f, __uint_as_float(o[e])));
                }
                tmem_st16(to + 16 * c, o);
            }
            tmem_st_wait();
        }
        if (ok) {
            const bool none = span[i].e <= span[i].s;         // no tile: O was never written
            // nor has a product shown that the row tile's other warps are done with the queries' place, which the outputs
            // go through: they meet first
            if (none) asm volatile("bar.sync %0, 128;" ::"r"(1 + i) : "memory");
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long all_rows = (long long)a.sq.tokens * a.heads, row = tok * a.heads + hrow;
            const bool part = rg.parts > 1;
            const float f = part ? 1.f : inv;
            // through shared memory (the queries' place, whose products are complete), so that rows are stored whole:
            // D 16-bit values or D/2 f32 values of each row at a time
            const bool wide = part || ot == MMQ_F32;
            const uint32_t stage = sb + C::q_off + i * C::kQBytes + (warp & 3) * (32 * D * 2);
            const long long mine = part ? (split * all_rows + row) * D * 4
                                        : (tok * a.out.ts + hrow * a.out.hs) * (ot == MMQ_F32 ? 4 : 2);
            uint8_t* dst = (part ? reinterpret_cast<uint8_t*>(a.part_o) : static_cast<uint8_t*>(a.out.data)) + sub * 16;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += wide ? D / 2 : D) {
#pragma unroll 4
                for (int c = 0; c < (wide ? D / 32 : D / 16); c++) {              // 16 columns
                    uint32_t o[16];
                    if (!none) {
                        tmem_ld16(to + d0 + 16 * c, o);
                        tmem_ld_wait(o);
                    }
                    float x[16];
#pragma unroll
                    for (int e = 0; e < 16; e++) {            // column order 0 2 1 3 undone
                        const int d = (e & ~3) | ((e & 1) << 1) | ((e >> 1) & 1);
                        x[d] = none || f == 0.f ? 0.f : __uint_as_float(o[e]) * f;
                    }
                    const uint32_t at = stage + lane * (D * 2);
                    if (wide) {
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            st_shared_v4(at + (((4 * c + k) ^ (lane & 7)) << 4), __float_as_uint(x[4 * k]),
                                         __float_as_uint(x[4 * k + 1]), __float_as_uint(x[4 * k + 2]),
                                         __float_as_uint(x[4 * k + 3]));
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                y[e] = ot == MMQ_BF16 ? pack2(x[8 * k + 2 * e], x[8 * k + 2 * e + 1], __nv_bfloat16())
                                                      : pack2(x[8 * k + 2 * e], x[8 * k + 2 * e + 1], __half());
                            st_shared_v4(at + (((2 * c + k) ^ (lane & 7)) << 4), y[0], y[1], y[2], y[3]);
                        }
                    }
                }
                __syncwarp();
#pragma unroll 8
                for (int s0 = 0; s0 < 32; s0 += RPS) {
                    const int at = s0 + lane / LPR;
                    const long long to_row = __shfl_sync(0xffffffffu, mine, at);
                    if ((r & ~31) + at < rows)
                        *reinterpret_cast<uint4*>(dst + to_row + (wide ? 4 * d0 : 0)) =
                            ld_shared_u4(stage + at * (D * 2) + ((sub ^ (at & 7)) << 4));
                }
                __syncwarp();
            }
            if (real) {
                if (part) a.part_ml[split * all_rows + row] = make_float2(l == 0.f ? -INFINITY : m, l);
                else if (a.lse) a.lse[row] = l == 0.f ? -INFINITY : LN2 * (m + log2f(l));
            }
        }
    }

    }
    // ---- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == T_MMA) tmem_dealloc(tmem, C::kCols);
}

template <int D, bool PACKED, bool LONG>
cudaError_t launch_tiled(long long slots, long long blocks, mmq_dtype qt, mmq_dtype ot, const AttnArgs& a,
                         const AttnPlan& p, cudaStream_t s) {
    const long long grid = blocks * a.c.heads * p.splits;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    auto kern = tiled_kernel<D, PACKED, LONG>;
    static bool configured[64] = {};
    bool& done = device_flag(configured);
    if (!done) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Tiled<D>::alloc);
        if (e != cudaSuccess) return e;
        done = true;
    }
    return launch_pdl_smem(kern, dim3((unsigned)grid), dim3(T_THREADS), Tiled<D>::alloc, s, a, p.chunk, (int)slots, (int)qt,
                           (int)ot);
}

// As many row blocks for every sequence as the longest needs, or, where that is more than twice as many as the packed rows
// need, blocks numbered through these.  An empty block costs an SM 2 us; the search of the packed form costs the tile loop
// 5 % (its values are no longer known to be uniform).  Four prompts of 1896 to 4096 tokens: 311 us, 328 packed; one of 2048
// with 63 single tokens: 239 us, 148 packed.
template <int D>
cudaError_t launch_tiled_rows(mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    constexpr int ROWS = 128 * Tiled<D>::kQTiles;
    const long long each = ((long long)a.max_tokens * a.group + ROWS - 1) / ROWS, all = each * a.sq.seqs;
    const long long packed = (long long)a.sq.tokens * a.group / ROWS + a.sq.seqs;
    // Parts that no sum has to be put aside in have a kernel without that code: prompts 306 us, 313 with it.
    const bool by_rows = a.sq.cu && all > 2 * packed, longer = p.chunk > kChain;
    const long long slots = by_rows ? packed : each, blocks = by_rows ? packed : all;
    auto launch = by_rows ? (longer ? launch_tiled<D, true, true> : launch_tiled<D, true, false>)
                          : (longer ? launch_tiled<D, false, true> : launch_tiled<D, false, false>);
    return launch(slots, blocks, qt, ot, a, p, s);
}

}  // namespace

cudaError_t run_attention_tiled(int dim, mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p,
                                cudaStream_t s) {
    switch (dim) {
        case 64: return launch_tiled_rows<64>(qt, ot, a, p, s);
        case 128: return launch_tiled_rows<128>(qt, ot, a, p, s);
        case 256: return launch_tiled_rows<256>(qt, ot, a, p, s);
    }
    return cudaErrorInvalidValue;
}

MMQ_DEFINE_ERROR_READER(attn_tiled)

}  // namespace mmq
