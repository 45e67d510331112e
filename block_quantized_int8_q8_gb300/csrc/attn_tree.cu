// attn_tree.cu -- attention of a tree's rows over the 8-bit paged cache, on tcgen05.
//
//   t_j = scale log2(e) ks_b (q . k_j) + log2(vs_b),  p_j = 2^(t_j - m),  O = sum_j p_j v_j,  l = sum_b (1/vs_b) sum_{j in b} p_j
//   out = O / l,  lse = ln(2) (m + log2 l)                (the formulas of attn_few.cu) over the j that a row sees
//
// For 17 to 128 rows (tokens x query heads of a group) of a sequence and key/value head: too many for mma.sync, and too few to
// fill the 128 lanes of a product whose rows they are, twice.  So the products stand the other way round, cache tokens and head
// dimensions on the 128 lanes and the query rows along the columns, of which there are R = 64 or 128:
//   S^T [128 tokens x R] = K Q^T       K: fp16 codes in TMEM (A operand), Q: shared memory, K-major
//   O^T [128 dims x R]  += V^T P^T     V: shared memory [token][64 dims of 128 bytes], M-major, P the same way, N-major
// A thread of the softmax then owns a token, with its scales in registers, and 32 of the rows; a group of rows that there are
// not costs nothing.  K never passes through shared memory, whose bandwidth is the next bound after the cache's.
//
// One thread block an SM.  The cache tiles of all (sequence, key/value head) units stand in one line, and each block takes an
// equal share of it, wherever that begins and ends (lengths are on the device: the blocks work out the line by themselves);
// units that are cut leave parts in the workspace, which a second launch joins.  Roles:
//   * groups of four softmax warps, each 32 of the rows: a tile's S^T, the mask, the exponentials, P as fp16 to shared memory.
//     The reference m of a row is raised only when a term passes it by 2^LAZY, which a group votes on; then O is rescaled.
//     They also list the block's share, bring the queries in and the results out.
//   * four warps turn the codes of K into fp16 in TMEM and seven (R = 128: three) those of V into shared memory, 32 tokens at
//     a time; the next codes are on their way to the registers that the last ones leave, those after them to L2.
//   * one warp issues the products, S up to kBufs tiles ahead.
// Bound by the latencies between the roles and, next, by instructions: a tile of 128 tokens of heads of 128 takes a block 1170 ns
// with 64 rows, where its codes take 737 at the rate of a plain copy; the converters alone take 896, the softmax alone 804, the
// products alone 550.  With 128 rows: 1573; 1318, 1096, 657.  Some 15 us of a call are its start, the first codes and the join.
// 16 sequences of 8192 tokens, 32 query and 8 key/value heads of 128: 85 us with 32 rows (3.2 TB/s), 92 with 64, 123 with 128
// (0.56 PFLOP/s); one of 131072, 64 rows, 90; 4 key/value heads of 256, 16 of 4000, 64 rows, 58.
// Slower: six warps for V (64 rows: 93 -> 102), eleven of fewer registers (96), eight for K (95).  Without any load of codes it
// would take 89 instead of 91: what is left is between the conversion, the softmax and the products, not memory.
#include <algorithm>
#include <type_traits>
#include "attn_device.cuh"
#include "attn_math.cuh"
#include "internal.h"

namespace mmq {

namespace {

constexpr int KT = 128;                      // cache tokens of a tile
constexpr int N = 32;                        // columns of a softmax group
constexpr int WINDOW = kChain / KT;          // most tiles that are listed, and summed, in one go
constexpr int RANGES = 152;                  // shares of the line of tiles: one a multiprocessor
constexpr float UNSET = 1e30f;               // -m of a row that has seen nothing yet

// Bit c of lane r becomes bit r of lane c: squares off the diagonal change places, ever smaller ones.
__device__ __forceinline__ uint32_t transpose32(uint32_t x, int lane) {
    uint32_t m = 0x0000FFFFu;
#pragma unroll
    for (int j = 16; j > 0; j >>= 1, m ^= m << j) {
        const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
        x = lane & j ? (x & ~m) | (y & ~m) >> j : (x & m) | (y & m) << j;
    }
    return x;
}

template <int D, int R> struct Tree {
    // warps of the converters and the products, after those of the softmax
    static constexpr int kGroups = R / N, kSoftmaxWarps = 4 * kGroups, kWarpsV = R == 128 ? 3 : 7;
    static constexpr int kWarpK = kSoftmaxWarps, kWarpV = kWarpK + 4, kWarpMma = kWarpV + kWarpsV, kWarps = kWarpMma + 1;
    static constexpr int kThreads = kWarps * 32;
    // Units that a converter warp has on their way to L2 besides those in its registers, one, two, three: 16 sequences of 8192, 32
    // rows, 83, 85, 88 us, 64 rows 91, 91, 95; 32 heads of 64, 16 of 2000, 64 rows, 99, 97, 97; heads of 256 61, 58, 60; with
    // 128 rows, where fewer registers are left, 123, 134 and 142.
    static constexpr int kAhead = R == 64 ? 2 : 1;
    // registers a thread: 20 warps have 96; of 24 each gets 80 at launch, some of which move to the softmax warps
    static constexpr int kRegsSoftmax = 88, kRegsRest = 64;
    static_assert(R == 64 || kSoftmaxWarps * kRegsSoftmax + 8 * kRegsRest <= 24 * 80, "register budget");
    static constexpr int kHalves = D == 256 ? 2 : 1;                             // O^T of 128 dimensions
    static constexpr int kStrips = D == 256 ? 2 : 1, kChunks = D == 64 ? 1 : 2;   // of up to 128 dimensions, of 64 each
    static constexpr int kVBytes = KT * D * 2, kQBytes = R * D * 2, kPBytes = KT * R * 2;
    static constexpr int kScaleSlots = 16;
    static constexpr int kKCols = D / 2;
    // Tiles of K and V that the converters may be ahead, three of V, two, two of each: 16 sequences of 8192, 32 rows, 85, 87, 86 us,
    // 64 rows 92, 93, 93, 128 rows 123, 120, 120; 64 sequences of 2000, 32 rows: 116, 120, 118.  32 heads of 64, 16 of 2000, 64
    // rows, four of V 97, three 101.
    static constexpr int kKStages = D == 64 ? 4 : (R == 64 && D == 128 ? 4 : 2);
    static constexpr int kVStages = D == 64 ? 4 : (D == 128 ? 3 : 2);
    // Buffers of S and of P.  With two, S of a tile waits for the softmax two tiles before, and then for the products in
    // between (two, three: 64 sequences of 2000, 32 rows, 120 and 116 us; 32 heads of 64, 16 of 2000, 64 rows, 101 and 97; 16
    // sequences of 8192, 64 rows, 93 and 92).
    static constexpr int kBufs = R == 64 && D <= 128 ? 3 : 2;
    // TMEM columns: S, O, K
    static constexpr int kOCol = kBufs * R, kKCol = kOCol + kHalves * R;
    static_assert(kKCol + kKStages * kKCols <= 512, "TMEM budget");
    // V first: for head_dim 64 the products read the next 16 KB as 64 more dimensions, whose results nothing looks at
    static constexpr int v_off = 0;
    static constexpr int q_off = v_off + kVStages * kVBytes;
    static constexpr int p_off = q_off + kQBytes;
    static constexpr int sc_off = p_off + kBufs * kPBytes;                           // float4 [slots][8]
    static constexpr int bar_off = sc_off + kScaleSlots * 8 * 16;
    static constexpr int n_bars = 3 + 3 * kBufs + 2 * (kKStages + kVStages);
    static constexpr int misc_off = bar_off + n_bars * 8;
    static constexpr int total = misc_off + 16, alloc = total + 1024;
    static_assert(alloc <= 232448 - (R == 64 ? 16 : 20) * 1024, "shared memory budget (the rest is static)");
};

// A run of tiles of one unit (sequence, key/value head, row block) in the block's share.
struct Piece {
    int s, head, n0;             // n0: first packed row of the sequence
    int first, lim;              // cached tokens before the new ones; tokens past lim do not exist
    int rows;
    int tok0;                    // first token of the run
    int x0, tiles;
    int slot;                    // its place in the workspace
    int flags;
};
constexpr int P_PREV = 1;        // continues what an earlier window left in the slot
constexpr int P_DIRECT = 2;      // ends the unit, of which no other block has a part

struct TreeWork {                // the workspace
    float* part_o;               // [2 ranges][R][D]
    float2* part_ml;             // [2 ranges][R]
    int4* joins;                 // [ranges][2]
};

__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
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
// 16 lanes x 32 columns in the layout of tmem_ld_16x256b_x4.
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptors as two words: the upper one (8-row groups 1024 bytes apart, 128-byte swizzle) is the
// same for all operands, the lower one holds start / 16 and, where M or N runs along the rows, the distance / 16 of its next 64.
constexpr uint32_t DESC_HI = (uint32_t)(((uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61) >> 32);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading) {
    return ((saddr & 0x3FFFFu) >> 4) | (leading >> 4) << 16;
}
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
// As mbar_wait, the first look without its loop.
__device__ __forceinline__ bool wait_for(uint32_t b, uint32_t parity, volatile int* abort_flag) {
    if (__builtin_expect(mbar_try_wait(b, parity), 1)) return true;
    return mbar_wait(b, parity, abort_flag);
}
// Whether any of the 128 threads at named barrier `id` says so.
__device__ __forceinline__ bool group_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "barrier.cta.red.or.pred p, %1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }
// 32 values of each lane, joined over the warp: lane c gets the result of the c-th.
template <bool MAX>
__device__ __forceinline__ float across(float (&x)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < o; i++) {
            const bool up = lane & o;
            const float keep = up ? x[i + o] : x[i], give = up ? x[i] : x[i + o];
            const float got = __shfl_xor_sync(0xffffffffu, give, o);
            x[i] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
    return x[0];
}

template <int D, int R> struct TreeBars {
    using C = Tree<D, R>;
    uint32_t b;
    __device__ uint32_t rest(int i) const { return b + 8u * i; }
    __device__ uint32_t qfull() const { return rest(0); }                        // a piece's queries
    __device__ uint32_t ofree() const { return rest(1); }                        // a piece's O is read
    __device__ uint32_t done() const { return rest(2); }
    // Of tiles i mod kBufs.  As products complete in their order, S of a tile shows that the product with V kBufs tiles before is
    // complete; pvdone has as many barriers, so that who has seen S of tile y may wait for the product of y or y - 1 without
    // having waited for those before: of that barrier, the phase before is over.
    __device__ uint32_t sfull(int i) const { return rest(3 + i); }
    __device__ uint32_t pready(int i) const { return rest(3 + C::kBufs + i); }
    __device__ uint32_t pvdone(int i) const { return rest(3 + 2 * C::kBufs + i); }
    __device__ uint32_t kfull(int i) const { return rest(3 + 3 * C::kBufs + i); }
    __device__ uint32_t kempty(int i) const { return rest(3 + 3 * C::kBufs + C::kKStages + i); }
    __device__ uint32_t vfull(int i) const { return rest(3 + 3 * C::kBufs + 2 * C::kKStages + i); }
    __device__ uint32_t vempty(int i) const { return rest(3 + 3 * C::kBufs + 2 * C::kKStages + C::kVStages + i); }
};

// What a unit costs besides its tiles, in tiles: its queries, its result, and the pipeline in between.  In the line it stands
// before them, or a block whose share lies among short sequences would be the last by far: 24 sequences of up to 8192 tokens,
// 64 rows, take 138 us with 0, 91 with 4, 87 with 5, 87 with 8; 16 of 8192 each, 32 rows, 86, 86, 85 and 88.
constexpr int EXTRA = 5;

// A sequence's place in the line of tiles.
struct Line {
    Seq q;
    int n, base;                 // new tokens, first token of the first tile
    int tiles;                   // of a unit
};
__device__ __forceinline__ Line line_of(const TreeArgs& a, int s) {
    Line x;
    x.q = load_seq(a.sq, s, a.c.page);
    x.n = min(x.q.n, a.max_tokens);
    const int first = x.q.len - x.q.n, lim = min(min(x.q.end, a.max_kv), first + x.n);
    x.base = a.window > 0 ? max(first - a.window + 1, 0) / 16 * 16 : 0;
    x.tiles = max((lim - x.base + KT - 1) / KT, 1);
    return x;
}

// The line of tiles: every sequence's units (its key/value heads) one after the other, shared out evenly.  The host keeps it
// below 2^30.
struct LineShare {
    int w[32], u[32];            // of the scan
    int span[2];                 // first and last unit with tiles in the window
    int skip, tiles;             // what the window has of the first one's EXTRA; the window's tiles
    int all, ranges;             // length of the line; shares that are not empty
    __device__ int start(int c) const { return c * (all / ranges) + min(c, all % ranges); }
    __device__ int range_of(int t) const {
        const int q = all / ranges, r = all % ranges;
        return t < r * (q + 1) ? t / (q + 1) : r + (t - r * (q + 1)) / q;
    }
};

// Lists the pieces of window `window` of this block's share; its first THREADS threads take part.  The first call works out
// the line.
template <int THREADS>
__device__ __forceinline__ void list_pieces(const TreeArgs& a, const TreeWork& work, LineShare& sh, Piece* pieces, int window) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = THREADS / 32, range = blockIdx.x;
    auto exclusive = [&](int w, int u, int& wx, int& ux, int& wall, int& uall) {
        int wi = w, ui = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, wi, o), z = __shfl_up_sync(0xffffffffu, ui, o);
            if (lane >= o) {
                wi += v;
                ui += z;
            }
        }
        named_bar_sync(15, THREADS);                          // the arrays' last readers are done
        if (lane == 31) {
            sh.w[warp] = wi;
            sh.u[warp] = ui;
        }
        named_bar_sync(15, THREADS);
        // every warp joins the warps' sums for itself
        int wv = lane < warps ? sh.w[lane] : 0, uv = lane < warps ? sh.u[lane] : 0;
        const int wm = wv, um = uv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, wv, o), z = __shfl_up_sync(0xffffffffu, uv, o);
            if (lane >= o) {
                wv += v;
                uv += z;
            }
        }
        wx = wi - w + __shfl_sync(0xffffffffu, wv - wm, warp);
        ux = ui - u + __shfl_sync(0xffffffffu, uv - um, warp);
        wall = __shfl_sync(0xffffffffu, wv, 31);
        uall = __shfl_sync(0xffffffffu, uv, 31);
    };
    Line x{};
    int w = 0, units = 0, wx = 0, ux = 0, wall = 0, uall = 0;
    auto look = [&](int s0) {
        const int s = s0 + threadIdx.x;
        w = units = 0;
        x = Line{};
        if (s < a.sq.seqs) {
            x = line_of(a, s);
            units = x.n > 0 ? a.c.heads : 0;
            w = (EXTRA + x.tiles) * units;
        }
        exclusive(w, units, wx, ux, wall, uall);
    };
    if (window == 0) {
        int all = 0;
        for (int s0 = 0; s0 < a.sq.seqs; s0 += THREADS) {
            look(s0);
            all += wall;
            const int s = s0 + threadIdx.x;
            if (range == 0 && s < a.sq.seqs) {
                const bool odd = a.sq.cu && odd_offsets(a.sq, s, a.sq.cu[s], a.sq.cu[s + 1]);
                if (odd || (x.n > 0 && (x.q.n > x.n || min(x.q.end, a.max_kv) < x.q.len))) flag_error(DEVERR_LENGTH);
            }
        }
        if (threadIdx.x == 0) {
            sh.all = all;
            sh.ranges = max(min((int)gridDim.x, all), 1);
        }
        named_bar_sync(15, THREADS);
    }
    if (range >= sh.ranges || sh.all == 0) {
        if (threadIdx.x == 0) work.joins[2 * range + 1] = make_int4(0, 0, 0, 0);
        return;
    }
    const int g0 = sh.start(range), g1 = sh.start(range + 1), g = g0 + window * WINDOW, gz = min(g + WINDOW, g1);
    if (g >= g1) return;
    const bool once = a.sq.seqs <= THREADS;                // what the first pass saw is still there
    int wbase = 0, ubase = 0;
    for (int s0 = 0; wbase < gz; s0 += THREADS) {
        if (!once || window > 0) look(s0);
        const int ws = wbase + wx, us = ubase + ux, each = EXTRA + x.tiles, s = s0 + threadIdx.x;
        if (ws <= g && g - ws < w) {
            const int k = (g - ws) / each, tile0 = ws + k * each + EXTRA;
            sh.span[0] = us + k;
            sh.skip = max(tile0 - g, 0);
            if (window == 0) {
                // The join of the unit that this range begins within, if the range before is the first with tiles of it.
                int parts = 0, slot0 = 0;
                if (tile0 < g && tile0 >= sh.start(range - 1)) {
                    parts = sh.range_of(tile0 + x.tiles - 1) - (range - 1) + 1;
                    slot0 = 2 * (range - 1) + (tile0 > sh.start(range - 1));
                }
                work.joins[2 * range] = make_int4(x.q.n0, x.n * a.group, k, 0);
                work.joins[2 * range + 1] = make_int4(parts, slot0, 2 * range, 0);
            }
        }
        named_bar_sync(15, THREADS);
        if (ws < gz && g - ws < w) {
            const int u0 = sh.span[0], first = x.q.len - x.q.n;
            const int k1 = min((gz - 1 - ws) / each, units - 1);
            for (int k = g > ws ? (g - ws) / each : 0; k <= k1; k++) {
                const int tile0 = ws + k * each + EXTRA, end = tile0 + x.tiles, lo = max(tile0, g), hi = min(end, gz);
                const int at = us + k - u0, x0 = at == 0 ? 0 : tile0 - g - sh.skip - at * EXTRA;
                if (end >= gz) {                              // the window's last, perhaps without tiles in it
                    sh.tiles = x0 + max(hi - lo, 0);
                    sh.span[1] = us + k - (hi <= lo);
                }
                if (hi <= lo) continue;
                Piece p;
                p.s = s;
                p.head = k;
                p.n0 = x.q.n0;
                p.first = first;
                p.lim = min(min(x.q.end, a.max_kv), first + x.n);
                p.rows = x.n * a.group;
                p.tok0 = x.base + (lo - tile0) * KT;
                p.x0 = x0;
                p.tiles = hi - lo;
                p.slot = 2 * range + (tile0 > g0);
                p.flags = (lo > max(tile0, g0) ? P_PREV : 0) | (hi == end && tile0 >= g0 ? P_DIRECT : 0);
                pieces[at] = p;
            }
        }
        wbase += wall;
        ubase += uall;
    }
}

template <int D, int R>
__global__ void __launch_bounds__(Tree<D, R>::kThreads, 1)
    tree_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ TreeWork work, int qt, int ot) {
    using C = Tree<D, R>;
    constexpr int STRIPS = C::kStrips, CU = C::kChunks, AHEAD = C::kAhead;
    pdl_wait();
    pdl_trigger();                                            // after the wait: the join reads its inputs before its own
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Piece s_piece[WINDOW];
    __shared__ LineShare s_line;
    __shared__ long long s_out[R];
    __shared__ int s_tok[R], s_low[R];
    __shared__ __align__(16) float s_neg[R], s_next[R];       // -m; largest magnitude of a query
    __shared__ float s_even[R];                               // what a row's S is to be multiplied by before the rest
    __shared__ float s_m[R], s_fac[R], s_add[R], s_red[C::kGroups][4][N];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sb = smem_u32(smem);
    const TreeBars<D, R> bar{sb + C::bar_off};
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc_off + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc_off);
    float4* scales = reinterpret_cast<float4*>(smem + C::sc_off);
    if (warp == C::kWarpMma) {
        if (lane == 0) {
            for (int i = 0; i < C::kKStages; i++) {
                mbar_init(bar.kfull(i), 4 * STRIPS);
                mbar_init(bar.kempty(i), 1);
            }
            for (int i = 0; i < C::kVStages; i++) {
                mbar_init(bar.vfull(i), 4 * STRIPS);
                mbar_init(bar.vempty(i), 1);
            }
            for (int i = 0; i < C::kBufs; i++) {
                mbar_init(bar.sfull(i), 2);                   // the product, and the thread that saw K and its scales
                mbar_init(bar.pready(i), C::kSoftmaxWarps);
                mbar_init(bar.pvdone(i), 1);
            }
            mbar_init(bar.qfull(), C::kSoftmaxWarps);
            mbar_init(bar.ofree(), C::kSoftmaxWarps);
            mbar_init(bar.done(), 1);
            *abort_flag = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    // Every role goes over the windows, which the softmax warps list; all meet when one is listed and when it is done.  The roles
    // stand inside the branch that sets their share of registers.
    auto windows = [&](auto lists, auto&& role) {
        int y0 = 0, k0 = 0;                                   // tiles and pieces of the windows before
#pragma unroll 1
        for (int window = 0;; window++) {
            if constexpr (decltype(lists)::value) list_pieces<32 * C::kSoftmaxWarps>(a, work, s_line, s_piece, window);
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            if (blockIdx.x >= s_line.ranges || s_line.start(blockIdx.x) + window * WINDOW >= s_line.start(blockIdx.x + 1)) break;
            const uint32_t tmem = *tmem_slot;
            const int tiles = s_line.tiles, pieces = s_line.span[1] - s_line.span[0] + 1;
            if (tiles > 0) role(tmem, tiles, pieces, y0, k0);       // (a share may lie between the tiles of two units)
            __syncthreads();
            y0 += tiles;
            k0 += pieces;
            if (*abort_flag) break;                           // (nothing waits here: the same for all)
        }
    };
    if (warp >= C::kWarpK) {
        if constexpr (R == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
        windows(std::false_type{}, [&](const uint32_t tmem, const int tiles, const int pieces, const int y0, const int k0) {
        if (warp != C::kWarpMma) {
            // ======================================================= converters
            // Units of 32 tokens (two groups of 16, each within one page and scale block) and up to 128 dimensions.  Of K, a warp
            // takes the quarter of a tile whose lanes of TMEM it can reach; of V, the warps take turns.  Lane (g, t) turns rows
            // g, g+8 of a group, 16 bytes at 16t of each 64.
            auto units_of = [&](auto side) {
                constexpr bool isv = decltype(side)::value;
                constexpr int TURN = isv ? C::kWarpsV : STRIPS;
                const int gr = lane >> 2, t = lane & 3, w = isv ? warp - C::kWarpV : warp - C::kWarpK;
                // the warp's u-th unit: tile, quarter of it, strip of 128 dimensions
                auto number = [&](int u) { return isv ? w + TURN * u : (u / STRIPS * 4 + w) * STRIPS + u % STRIPS; };
                const int units = isv ? (4 * STRIPS * tiles - w + TURN - 1) / TURN : STRIPS * tiles;
                const int8_t* codes = (isv ? a.c.v : a.c.k) + gr * D + 16 * t;
                // lanes 2i, 2i+1: the groups of the i-th of the warp's next 16 units: place / 16, and the scales.  Where there is
                // nothing, any codes will do: the score's factor and iv are zero, and so is the probability.
                int src = 0;
                float ks = 0.f, lv = -INFINITY, iv = 0.f;
                auto lookup = [&](int u0) {
                    const int u = u0 + (lane >> 1), v = number(u), x = v / (4 * STRIPS);
                    src = 0, ks = 0.f, lv = -INFINITY, iv = 0.f;
                    if (u >= units) return;
                    int lo = 0, hi = pieces;                  // the piece that tile x lies in
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) / 2;
                        if (s_piece[mid].x0 <= x) lo = mid;
                        else hi = mid;
                    }
                    const Piece& p = s_piece[lo];
                    const int tok = p.tok0 + (x - p.x0) * KT + 32 * (v / STRIPS & 3) + 16 * (lane & 1);
                    if (tok >= p.lim) return;
                    const int page = tok / a.c.page, off = tok - page * a.c.page;
                    const int pg = a.sq.table[p.s * a.sq.stride + page];
                    if ((unsigned)pg < (unsigned long long)a.c.pages) {
                        const int ph = pg * a.c.heads + p.head;
                        src = ph * (a.c.page / 16) + off / 16;
                        if constexpr (!isv) {
                            const long long sc = (long long)ph * (a.c.page / a.c.block) + off / a.c.block;
                            ks = a.c.ks[sc];
                            const float vs = fmaxf(a.c.vs[sc], SCALE_FLOOR);
                            lv = __log2f(vs);
                            iv = __fdividef(1.f, vs);
                        }
                    } else {
                        flag_error(DEVERR_PAGE);
                    }
                };
                // Places of the next AHEAD units, whose codes are on their way to the L2 cache: from there they come in half
                // the time that memory takes, and a warp holds no more than one unit's loads.
                int place[AHEAD][2];
                auto step = [&](int u) {                      // unit u's place goes into the queue, its scales to the softmax
                    if ((u & 15) == 0) lookup(u);
#pragma unroll
                    for (int i = 0; i + 1 < AHEAD; i++)
#pragma unroll
                        for (int g = 0; g < 2; g++) place[i][g] = place[i + 1][g];
#pragma unroll
                    for (int g = 0; g < 2; g++) place[AHEAD - 1][g] = __shfl_sync(0xffffffffu, src, 2 * (u & 15) + g);
                    const int strip = number(u) % STRIPS;
                    if (u >= units) return;
                    // lane -> a row's codes of the strip, 128 bytes at most
                    prefetch_l2((isv ? a.c.v : a.c.k) + (long long)(lane < 16 ? place[AHEAD - 1][0] : place[AHEAD - 1][1]) * (16 * D) +
                                (lane & 15) * D + 128 * strip);
                    // (the slot's last readers are behind: K is at most kKStages + kBufs tiles ahead of the softmax, this AHEAD more)
                    if (!isv && (lane >> 1) == (u & 15) && strip == 0)
                        scales[(y0 + u / STRIPS) % C::kScaleSlots * 8 + 2 * w + (lane & 1)] = make_float4(ks, lv, iv, 0.f);
                };
                static_assert(C::kKStages + C::kBufs + AHEAD < C::kScaleSlots, "scale slots");
                const int8_t* from[2];
                auto point = [&](int u) {                     // at unit u's codes, the queue's first
                    const int strip = number(u) % STRIPS;
#pragma unroll
                    for (int g = 0; g < 2; g++) from[g] = codes + (long long)place[0][g] * (16 * D) + 128 * strip;
                };
                // A barrier shows a phase's parity only, so a warp must not be two phases off.  It is not lapped, since its own
                // unit completes the tile; and as stages are released in the order of the tiles, the wait for its unit before,
                // at most a lap of stages back, shows that the phase before this one is complete.
                static_assert((TURN + 4 * STRIPS - 1) / (4 * STRIPS) <= (isv ? C::kVStages : C::kKStages), "units too far apart");
                uint4 r[2][2][CU];
#pragma unroll 1
                for (int u = 0; u < AHEAD; u++) step(u);
                point(0);
#pragma unroll
                for (int g = 0; g < 2; g++)
#pragma unroll
                    for (int h = 0; h < 2; h++)
#pragma unroll
                        for (int c = 0; c < CU; c++) r[g][h][c] = ld_cache(from[g] + 8 * h * D + 64 * c);
                bool ok = true;
#pragma unroll 1
                for (int u = 0; u < units; u++) {
                    step(u + AHEAD);
                    point(u + 1);
                    const int v = number(u), y = y0 + v / (4 * STRIPS), quarter = v / STRIPS & 3, strip = v % STRIPS;
                    const int st = y % (isv ? C::kVStages : C::kKStages);
                    const uint32_t full = isv ? bar.vfull(st) : bar.kfull(st);
                    ok = ok && mbar_wait_relaxed(isv ? bar.vempty(st) : bar.kempty(st),
                                                 ((y / (isv ? C::kVStages : C::kKStages)) & 1) ^ 1, abort_flag);
                    if constexpr (isv) {
                        const uint32_t to = sb + C::v_off + st * C::kVBytes + quarter * (32 * 128) + strip * (2 * KT * 128);
#pragma unroll
                        for (int g = 0; g < 2; g++)
#pragma unroll
                            for (int h = 0; h < 2; h++)
#pragma unroll
                                for (int c = 0; c < CU; c++) {
                                    const uint4 x = r[g][h][c];
                                    uint32_t z[8];
                                    codes_even_odd(x.x, z[0], z[1]);
                                    codes_even_odd(x.y, z[2], z[3]);
                                    codes_even_odd(x.z, z[4], z[5]);
                                    codes_even_odd(x.w, z[6], z[7]);
                                    r[g][h][c] = ld_cache(from[g] + 8 * h * D + 64 * c);
                                    const uint32_t place = to + c * (KT * 128) + g * 2048 + h * 1024;
                                    st_shared_v4(place + sw128_off(gr, 2 * t), z[0], z[1], z[2], z[3]);
                                    st_shared_v4(place + sw128_off(gr, 2 * t + 1), z[4], z[5], z[6], z[7]);
                                }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full);
                    } else {
                        tc_fence_after();
                        const uint32_t to = tmem + ((uint32_t)(32 * quarter) << 16) + C::kKCol + st * C::kKCols + 64 * strip;
#pragma unroll
                        for (int g = 0; g < 2; g++)
#pragma unroll
                            for (int c = 0; c < CU; c++) {
                                uint32_t z[16];
#pragma unroll
                                for (int h = 0; h < 2; h++) {
                                    const uint4 x = r[g][h][c];
                                    codes_even_odd(x.x, z[2 * h], z[2 * h + 1]);
                                    codes_even_odd(x.y, z[4 + 2 * h], z[4 + 2 * h + 1]);
                                    codes_even_odd(x.z, z[8 + 2 * h], z[8 + 2 * h + 1]);
                                    codes_even_odd(x.w, z[12 + 2 * h], z[12 + 2 * h + 1]);
                                    r[g][h][c] = ld_cache(from[g] + 8 * h * D + 64 * c);
                                }
                                tmem_st_16x256b_x4(to + ((uint32_t)(16 * g) << 16) + 32 * c, z);
                            }
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(full);
                        }
                    }
                }
            };
            if (warp >= C::kWarpV) units_of(std::true_type());
            else units_of(std::false_type());
        } else {
            // ======================================================= products
            constexpr uint32_t idesc_s = idesc_f16_f32(128, R);
            constexpr uint32_t idesc_o = idesc_f16_f32(128, R) | (1u << 15) | (1u << 16);     // M and N along the rows
            const uint32_t q_lo = desc_lo(sb + C::q_off, 16), v_lo = desc_lo(sb + C::v_off, KT * 128);
            const uint32_t p_lo = desc_lo(sb + C::p_off, KT * 128);
            bool ok = true;
            int ks = 0, kx = 0;                               // the piece whose S comes next, and its first tile
            auto product_s = [&](int x) {
                const int y = y0 + x;
                if (x == kx) {
                    ok = ok && wait_for(bar.qfull(), (k0 + ks) & 1, abort_flag);
                    ks++;
                    kx = ks < pieces ? s_piece[ks].x0 : tiles;
                }
                const int st = y % C::kKStages, buf = y % C::kBufs;
                ok = ok && wait_for(bar.kfull(st), (y / C::kKStages) & 1, abort_flag);
                if (!ok) return;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; k++)
                        umma_ts(tmem + buf * R, tmem + C::kKCol + st * C::kKCols + 8 * k,
                                q_lo + (k / 4) * (R * 128 >> 4) + 2 * (k % 4), idesc_s, k > 0);
                    mbar_arrive(bar.sfull(buf));
                    umma_commit(bar.sfull(buf));
                    umma_commit(bar.kempty(st));
                }
                __syncwarp();
            };
            int ko = 0, xo = 0;                               // the piece whose O is summed next, and its first tile
            int xs = 0;                                       // tile whose S comes next
            for (int x = 0; ok && x < tiles; x++) {
                const int y = y0 + x, buf = y % C::kBufs;
                // S is ahead of the softmax, but for a piece's first tile: its queries come after the last piece's last tile
                while (ok && xs < tiles && xs < x + C::kBufs && (xs != kx || xs == x)) product_s(xs++);
                const bool fresh = x == xo;
                if (fresh) {
                    if (k0 + ko > 0) ok = ok && wait_for(bar.ofree(), (k0 + ko - 1) & 1, abort_flag);
                    ko++;
                    xo = ko < pieces ? s_piece[ko].x0 : tiles;
                }
                const int st = y % C::kVStages;
                ok = ok && wait_for(bar.vfull(st), (y / C::kVStages) & 1, abort_flag);
                ok = ok && wait_for(bar.pready(buf), (y / C::kBufs) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t p = p_lo + buf * (C::kPBytes >> 4), v = v_lo + st * (C::kVBytes >> 4);
#pragma unroll
                    for (int h = 0; h < C::kHalves; h++)
#pragma unroll
                        for (int k = 0; k < KT / 16; k++)
                            umma_ss(tmem + C::kOCol + h * R, v + h * (2 * KT * 128 >> 4) + k * (2048 >> 4), p + k * (2048 >> 4),
                                    idesc_o, !fresh || k > 0);
                    umma_commit(bar.pvdone(buf));
                    umma_commit(bar.vempty(st));
                }
                __syncwarp();
            }
        }
        });
        if (warp == C::kWarpMma) {
            if (elect_one()) umma_commit(bar.done());
            __syncwarp();
            mbar_wait_final(bar.done(), 0);
            __syncwarp();
        }
    } else {
        if constexpr (R == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
        windows(std::true_type{}, [&](const uint32_t tmem, const int, const int pieces, const int y0, const int) {
            // ======================================================= softmax: one thread a token
            // A failed wait does not leave the loops (the group meets at barriers); later waits then return at once.
            const int grp = warp >> 2, w = warp & 3, tk = 32 * w + lane, gt = threadIdx.x & 127, c0 = grp * N;
            const int id = 1 + grp;
            constexpr int LPR = D / 8, RPP = 4 * 32 / LPR;    // lanes on a row of queries, rows at a time
            const uint32_t lanes = (uint32_t)(32 * w) << 16;
            bool ok = true;
            auto fetch_q = [&](const Piece& p) {
                if (p.rows <= c0) return;
#pragma unroll
                for (int i = 0; i < N; i += RPP) {
                    const int c = c0 + i + (w * 32 + lane) / LPR, row = min(c, p.rows - 1), m = lane % LPR;
                    const uint16_t* from = static_cast<const uint16_t*>(a.q.data) + (long long)(p.n0 + row / a.group) * a.q.ts +
                                           (long long)(p.head * a.group + row % a.group) * a.q.hs + 8 * m;
                    cp_async_16(sb + C::q_off + (m / 8) * (R * 128) + sw128_off(c, m % 8), from, c < p.rows ? 16 : 0);
                }
                cp_async_commit();
            };
            // In place to fp16, in the order in which K's dimensions stand: group w of four dimensions of 16t .. 16t + 15 at place
            // 4w + t, 0 2 1 3 within.  All rows of the group by one power of two, which brings the largest magnitude to
            // [2^14, 2^15), so that one factor turns S into scores: a row is then exact where it was exact on its own, down
            // to 2^-14 of its largest value and rounded to 2^-25 of it below, as long as that is within 2^13 of the group's.
            // A smaller row is brought that near, and its S is multiplied by the rest (s_even) first.  So is a row so large
            // that the common factor would reach 1 (|scale q| from some 10^4 on): the factor times a key's scale is then finite
            // whatever the row, and a row out of bounds leaves its neighbours alone.
            float factor = 0.f;                               // of the next piece's scores
            bool uneven = false;
            auto convert_q = [&](const Piece& p) {
                if (p.rows > c0) {
                    const int m = lane % LPR;
                    const uint32_t panel = sb + C::q_off + (m / 8) * (R * 128);
                    cp_async_wait<0>();
#pragma unroll 1
                    for (int i = 0; i < N; i += RPP) {
                        const int c = c0 + i + (w * 32 + lane) / LPR;
                        float x[8], top = 0.f;
                        unpack8(ld_shared_u4(panel + sw128_off(c, m % 8)), qt == MMQ_BF16, x);
#pragma unroll
                        for (int e = 0; e < 8; e++) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
                        for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        if (m == 0) s_next[c] = top;
                    }
                    named_bar_sync(id, 128);
                    const float own = s_next[c0 + lane];      // (an infinite row is its own affair)
                    float most = own < INFINITY ? own : 0.f;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                    // exponents count from 127; a zero row's does not matter; up to cap the factor is below 1
                    const int cap = 267 - (int)(__float_as_uint(fabsf(a.scale * LOG2E)) >> 23);
                    const int high = min(max((int)(__float_as_uint(most) >> 23), 1), cap);
                    factor = a.scale * LOG2E * pow2((high - 141) / 2) * pow2(high - 141 - (high - 141) / 2);
                    uneven = false;
#pragma unroll 1
                    for (int i = 0; i < N; i += RPP) {
                        const int c = c0 + i + (w * 32 + lane) / LPR;
                        const float top = s_next[c];
                        const int e2 = max((int)(__float_as_uint(top) >> 23), 1);
                        const int rest = top == 0.f ? 0 : max(high - 13 - e2, 0) + min(high - e2, 0);
                        const int up = 141 - high + rest;
                        const float up0 = pow2(up / 2), up1 = pow2(up - up / 2);
                        float x[8];
                        unpack8(ld_shared_u4(panel + sw128_off(c, m % 8)), qt == MMQ_BF16, x);
#pragma unroll
                        for (int e = 0; e < 8; e++) x[e] = x[e] * up0 * up1;
                        const int half = min(max(-rest, -126), 127);
                        if (m == 0) s_even[c] = pow2(half) * pow2(-rest - half);
                        uneven |= rest != 0;
                        __syncwarp();                         // the rows are read
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int four = 2 * (m % 8) + e, place = 4 * (four & 3) + (four >> 2);
                            const uint32_t lo = pack2(x[4 * e], x[4 * e + 2], __half());
                            const uint32_t hi = pack2(x[4 * e + 1], x[4 * e + 3], __half());
                            asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(panel + sw128_off(c, place >> 1) + 8 * (place & 1)),
                                         "r"(lo), "r"(hi)
                                         : "memory");
                        }
                    }
                    uneven = group_any(id, uneven);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.qfull());
            };
            fetch_q(s_piece[0]);
            convert_q(s_piece[0]);
            for (int k = 0; k < pieces; k++) {
                const Piece& p = s_piece[k];
                const bool busy = p.rows > c0, more = k + 1 < pieces;
                named_bar_sync(id, 128);                      // the last piece's values are read
                if (gt < N) {
                    const int c = c0 + gt, row = min(c, p.rows - 1), tok = p.n0 + row / a.group;
                    const bool real = c < p.rows;
                    s_neg[c] = real ? UNSET : -INFINITY;
                    s_m[c] = -INFINITY;
                    s_tok[c] = tok;
                    if (a.window > 0) {
                        const int depth = a.depths[tok], held = tree_depth(depth, a.max_tokens);
                        if (held != depth) flag_error(DEVERR_DRAFT);
                        s_low[c] = p.first + held - a.window + 1;
                    }
                    s_out[c] = (long long)tok * a.out.ts + (p.head * a.group + row % a.group) * a.out.hs;
                }
                named_bar_sync(id, 128);
                uint64_t l2[N / 2];
#pragma unroll
                for (int i = 0; i < N / 2; i++) l2[i] = 0ull;
                // every row sees every token of the tiles from y_low to before y_high, between the window's edge and the new tokens
                // (or what the bounds leave of the cached ones)
                const int y_end = y0 + p.x0 + p.tiles;
                const int y_high = y0 + p.x0 + max(min(p.first, p.lim) - p.tok0, 0) / KT;
                const int y_low = a.window > 0 ? y0 + p.x0 + (max(p.first + a.max_tokens - a.window - p.tok0, -1) + KT) / KT : 0;
#pragma unroll 1
                for (int y = y0 + p.x0; y < y_end; y++) {
                    const int buf = y % C::kBufs;
                    const bool masked = y >= y_high || y < y_low;
                    uint32_t see[N / 32];
#pragma unroll
                    for (int b = 0; b < N / 32; b++) see[b] = 0xFFFFFFFFu;
                    if (__builtin_expect(masked && busy, 0)) {
                        // lane c: what column c sees of the warp's 32 tokens; turned over, so that a token has its columns
                        const int j0 = p.tok0 + (y - (y_end - p.tiles)) * KT + 32 * w;
#pragma unroll
                        for (int b = 0; b < N / 32; b++) {
                            const int c = c0 + 32 * b + lane, low = a.window > 0 ? s_low[c] - j0 : 0;
                            see[b] = transpose32(tree_sees(a.masks + (long long)s_tok[c] * a.words, a.words, j0 - p.first, low, p.lim - j0),
                                                 lane);
                        }
                    }
                    ok = wait_for(bar.sfull(buf), (y / C::kBufs) & 1, abort_flag) && ok;
                    tc_fence_after();
                    if (more && y + 1 == y_end) fetch_q(s_piece[k + 1]);                      // every S of the piece is complete
                    if (busy) {
                        const float4 sc = scales[y % C::kScaleSlots * 8 + tk / 16];
#pragma unroll
                        for (int b = 0; b < N / 32; b++) {    // 32 columns
                            const int cb = c0 + 32 * b;
                            uint32_t xr[32];
                            float e[32];
                            auto terms = [&](auto shifted) {  // e = t - m, or t
                                const uint64_t g2 = f2_pack(factor * sc.x, factor * sc.x), lv2 = f2_pack(sc.y, sc.y);
                                tmem_ld32(tmem + lanes + buf * R + cb, xr);
                                tmem_wait32(xr);
                                if (__builtin_expect(uneven, 0))
#pragma unroll
                                    for (int i = 0; i < 32; i++) xr[i] = __float_as_uint(__uint_as_float(xr[i]) * s_even[cb + i]);
#pragma unroll
                                for (int i = 0; i < 8; i++) {
                                    const float4 neg = reinterpret_cast<const float4*>(s_neg + cb)[i];
#pragma unroll
                                    for (int u = 0; u < 2; u++) {
                                        const uint64_t n2 = u ? f2_pack(neg.z, neg.w) : f2_pack(neg.x, neg.y);
                                        const uint64_t sh = decltype(shifted)::value ? f2_add(n2, lv2) : lv2;
                                        const int at = 4 * i + 2 * u;
                                        f2_unpack(f2_fma(f2_pack(__uint_as_float(xr[at]), __uint_as_float(xr[at + 1])), g2, sh), e[at],
                                                  e[at + 1]);
                                    }
                                }
                                if (__builtin_expect(masked, 0))
#pragma unroll
                                    for (int i = 0; i < 32; i++)
                                        if (!(see[b] >> i & 1u)) e[i] = -INFINITY;
                            };
#pragma unroll 1
                            for (int raised = 0;; raised++) {
                                terms(std::true_type());
                                float tops[4] = {max3(e[0], e[1], e[2]), max3(e[3], e[4], e[5]), max3(e[6], e[7], e[8]), fmaxf(e[9], e[10])};
#pragma unroll
                                for (int i = 11; i < 27; i += 8)
#pragma unroll
                                    for (int u = 0; u < 4; u++) tops[u] = max3(tops[u], e[i + 2 * u], e[i + 2 * u + 1]);
                                const float top = max3(max3(tops[0], tops[1], tops[2]), max3(tops[3], e[27], e[28]), max3(e[29], e[30], e[31]));
                                if (__builtin_expect(!group_any(id, top > LAZY) || raised, 1)) break;
                                // a term passes its row's reference by 2^LAZY: raise the references (once: then none does)
                                terms(std::false_type());
                                s_red[grp][w][32 * b + lane] = across<true>(e);
                                named_bar_sync(id, 128);
                                if (gt < 32) {
                                    const int c = cb + gt, at = 32 * b + gt;
                                    const float(&red)[4][N] = s_red[grp];
                                    const float most = fmaxf(fmaxf(red[0][at], red[1][at]), fmaxf(red[2][at], red[3][at]));
                                    const float m = s_m[c], mn = fmaxf(m, most - HEAD);
                                    s_fac[c] = m == -INFINITY ? 1.f : ex2(m - mn);
                                    if (c < p.rows && mn > -INFINITY) {
                                        s_m[c] = mn;
                                        s_neg[c] = -mn;
                                    }
                                }
                                named_bar_sync(id, 128);
                                const auto fac = [&](int i) { return f2_pack(s_fac[cb + 2 * i], s_fac[cb + 2 * i + 1]); };
#pragma unroll
                                for (int i = 0; i < 16; i++) l2[16 * b + i] = f2_mul(l2[16 * b + i], fac(i));
                                if (y > y_end - p.tiles) {
                                    ok = wait_for(bar.pvdone((y - 1) % C::kBufs), ((y - 1) / C::kBufs) & 1, abort_flag) && ok;
                                    tc_fence_after();
#pragma unroll 1
                                    for (int o = 0; o < 2 * C::kHalves; o++) {        // halves of the columns, dimensions
                                        const uint32_t at = tmem + lanes + C::kOCol + (o >> 1) * R + cb + 16 * (o & 1);
                                        uint32_t half[16];
                                        tmem_ld16(at, half);
                                        tmem_ld_wait(half);
#pragma unroll
                                        for (int i = 0; i < 16; i++)
                                            half[i] = __float_as_uint(__uint_as_float(half[i]) * s_fac[cb + 16 * (o & 1) + i]);
                                        tmem_st16(at, half);
                                    }
                                    tmem_st_wait();
                                }
                            }
                            // (P's buffer is free: S of this tile came after the product that read it)
                            const uint32_t row = sb + C::p_off + buf * C::kPBytes + (cb / 64) * (KT * 128);
                            const uint64_t iv2 = f2_pack(sc.z, sc.z);
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                uint32_t z[4];
#pragma unroll
                                for (int u = 0; u < 4; u++) {
                                    const float p0 = ex2(e[8 * i + 2 * u]), p1 = ex2(e[8 * i + 2 * u + 1]);
                                    l2[16 * b + 4 * i + u] = f2_fma(f2_pack(p0, p1), iv2, l2[16 * b + 4 * i + u]);
                                    z[u] = pack2(p0, p1, __half());
                                }
                                st_shared_v4(row + sw128_off(tk, cb % 64 / 8 + i), z[0], z[1], z[2], z[3]);
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar.pready(buf));
                }
                if (more) convert_q(s_piece[k + 1]);
                // ---- the piece's result
                const int yz = y_end - 1;
                ok = wait_for(bar.pvdone(yz % C::kBufs), (yz / C::kBufs) & 1, abort_flag) && ok;
                tc_fence_after();
                if (busy) {
#pragma unroll
                    for (int b = 0; b < N / 32; b++) {
                        float e[32];
#pragma unroll
                        for (int i = 0; i < 16; i++) f2_unpack(l2[16 * b + i], e[2 * i], e[2 * i + 1]);
                        s_red[grp][w][32 * b + lane] = across<false>(e);
                    }
                    named_bar_sync(id, 128);
                    if (gt < N && c0 + gt < p.rows) {
                        const int c = c0 + gt;
                        const float(&red)[4][N] = s_red[grp];
                        float l = red[0][gt] + red[1][gt] + (red[2][gt] + red[3][gt]), m = s_m[c], keep = 1.f, add = 0.f;
                        float2* ml = work.part_ml + (long long)p.slot * R + c;
                        if (p.flags & P_PREV) {
                            const float2 was = *ml;
                            const float both = fmaxf(was.x, m);
                            keep = m == -INFINITY ? 0.f : ex2(m - both);
                            add = was.x == -INFINITY ? 0.f : ex2(was.x - both);
                            l = fmaf(was.y, add, l * keep);
                            m = both;
                        }
                        if (p.flags & P_DIRECT) {
                            const float inv = l == 0.f ? 0.f : 1.f / l;
                            keep *= inv;
                            add *= inv;
                            if (ok && a.lse)
                                a.lse[(long long)s_tok[c] * a.heads + p.head * a.group + c % a.group] =
                                    l == 0.f ? -INFINITY : LN2 * (m + log2f(l));
                        } else if (ok) {
                            *ml = make_float2(m, l);
                        }
                        s_fac[c] = keep;
                        s_add[c] = add;
                    }
                    named_bar_sync(id, 128);
                    if (ok && (D != 64 || w < 2)) {
                        const int dim = 32 * w + ((lane & ~3) | (lane & 1) << 1 | (lane >> 1 & 1));       // order 0 2 1 3 undone
#pragma unroll 1
                        for (int b = 0; b < C::kHalves * (N / 16); b++) {
                            const int o = b / (N / 16), cb = c0 + b % (N / 16) * 16, d = 128 * o + dim;
                            uint32_t xr[16];
                            tmem_ld16(tmem + lanes + C::kOCol + o * R + cb, xr);
                            tmem_ld_wait(xr);
                            float* part = work.part_o + ((long long)p.slot * R + cb) * D + d;
                            const int left = p.rows - cb, flags = p.flags;
#pragma unroll
                            for (int i = 0; i < 16; i++) {
                                if (i >= left) break;
                                const float keep = s_fac[cb + i];
                                float v = keep == 0.f ? 0.f : __uint_as_float(xr[i]) * keep;
                                if (flags & P_PREV) v = fmaf(part[i * D], s_add[cb + i], v);
                                if (flags & P_DIRECT) {
                                    const long long at = s_out[cb + i] + d;
                                    if (ot == MMQ_F32) static_cast<float*>(a.out.data)[at] = v;
                                    else if (ot == MMQ_BF16) static_cast<__nv_bfloat16*>(a.out.data)[at] = __float2bfloat16(v);
                                    else static_cast<__half*>(a.out.data)[at] = __float2half(v);
                                } else {
                                    part[i * D] = v;
                                }
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.ofree());
            }
        });
    }
    // ---- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::kWarpMma) tmem_dealloc(*tmem_slot, 512);
}

// The parts of a unit that several ranges hold, on a common reference and in their order.  A block looks after rows of the
// unit that goes over the boundary before range `c`, where that is the unit's first; W warps a row.
template <int D, int W>
__global__ void __launch_bounds__(128) tree_join_kernel(const TreeArgs a, const TreeWork work, int R, int ot) {
    constexpr int ROWS = 4 / W, PER = D / 32;
    __shared__ float s_acc[W > 1 ? W : 1][W > 1 ? D : 1], s_den[W];
    const int per = R / ROWS, c = 1 + blockIdx.x / per, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x % per * ROWS + (W > 1 ? 0 : warp), w = W > 1 ? warp : 0;
    pdl_wait();
    const int4 parts = work.joins[2 * c + 1];
    if (parts.x == 0) return;
    const int4 unit = work.joins[2 * c];                      // first token, rows, head
    if (row >= unit.y) return;
    auto place = [&](int p) { return (long long)(p == 0 ? parts.y : parts.z + 2 * (p - 1)) * R + row; };
    float mx = -INFINITY;
    for (int p = lane; p < parts.x; p += 32) mx = fmaxf(mx, work.part_ml[place(p)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float acc[PER] = {}, den = 0.f;
#pragma unroll 4
    for (int p = w; p < parts.x; p += W) {
        const float2 ml = work.part_ml[place(p)];
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx);
        const float* from = work.part_o + place(p) * D + lane;
        den = fmaf(ml.y, f, den);
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const float v = from[32 * e];
            acc[e] = f == 0.f ? acc[e] : fmaf(v, f, acc[e]);
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < PER; e++) s_acc[w][lane + 32 * e] = acc[e];
        if (lane == 0) s_den[w] = den;
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int u = 1; u < W; u++) {
            den += s_den[u];
#pragma unroll
            for (int e = 0; e < PER; e++) acc[e] += s_acc[u][lane + 32 * e];
        }
    }
    const int h = unit.z * a.group + row % a.group;
    const long long tok = unit.x + row / a.group, at = tok * a.out.ts + h * a.out.hs + lane;
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const float v = inv == 0.f ? 0.f : acc[e] * inv;
        if (ot == MMQ_F32) static_cast<float*>(a.out.data)[at + 32 * e] = v;
        else if (ot == MMQ_BF16) static_cast<__nv_bfloat16*>(a.out.data)[at + 32 * e] = __float2bfloat16(v);
        else static_cast<__half*>(a.out.data)[at + 32 * e] = __float2half(v);
    }
    if (lane == 0 && a.lse) a.lse[tok * a.heads + h] = den == 0.f ? -INFINITY : LN2 * (mx + log2f(den));
}

template <int D, int R>
cudaError_t launch_tree(mmq_dtype qt, mmq_dtype ot, const TreeArgs& a, const TreePlan& p, void* ws, cudaStream_t s) {
    uint8_t* base = static_cast<uint8_t*>(ws);
    const TreeWork work{reinterpret_cast<float*>(base + p.part_o), reinterpret_cast<float2*>(base + p.part_ml),
                        reinterpret_cast<int4*>(base + p.joins)};
    auto kern = tree_kernel<D, R>;
    static bool configured[64] = {};
    bool& done = device_flag(configured);
    if (!done) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Tree<D, R>::alloc);
        if (e != cudaSuccess) return e;
        done = true;
    }
    cudaError_t e = launch_pdl_smem(kern, dim3(RANGES), dim3(Tree<D, R>::kThreads), Tree<D, R>::alloc, s, a, work, (int)qt,
                                    (int)ot);
    if (e != cudaSuccess) return e;
    if (p.many_parts)
        return launch_pdl(tree_join_kernel<D, 4>, dim3((unsigned)((RANGES - 1) * R)), dim3(128), s, a, work, R, (int)ot);
    return launch_pdl(tree_join_kernel<D, 1>, dim3((unsigned)((RANGES - 1) * (R / 4))), dim3(128), s, a, work, R, (int)ot);
}

}  // namespace

TreePlan tree_plan(int heads, int kv_heads, int dim, int seqs, long long max_tokens, long long max_kv) {
    TreePlan p{};
    p.rows = max_tokens * (heads / kv_heads) <= 64 ? 64 : 128;
    const long long units = (long long)kv_heads * seqs;
    p.fits = (double)units * (double)(EXTRA + max_kv / KT + 1) < 1073741824.0;
    p.many_parts = units <= RANGES / 8;
    size_t off = 0;
    p.joins = off;
    off += ((size_t)RANGES * 2 * sizeof(int4) + 255) & ~size_t(255);
    p.part_ml = off;
    off += ((size_t)RANGES * 2 * p.rows * sizeof(float2) + 255) & ~size_t(255);
    p.part_o = off;
    off += (size_t)RANGES * 2 * p.rows * dim * sizeof(float);
    p.total = off;
    return p;
}

cudaError_t run_attention_tree(int dim, mmq_dtype qt, mmq_dtype ot, const TreeArgs& a, const TreePlan& p, void* workspace,
                               cudaStream_t s) {
    switch (dim) {
        case 64: return p.rows == 64 ? launch_tree<64, 64>(qt, ot, a, p, workspace, s)
                                     : launch_tree<64, 128>(qt, ot, a, p, workspace, s);
        case 128: return p.rows == 64 ? launch_tree<128, 64>(qt, ot, a, p, workspace, s)
                                      : launch_tree<128, 128>(qt, ot, a, p, workspace, s);
        case 256: return launch_tree<256, 64>(qt, ot, a, p, workspace, s);
    }
    return cudaErrorInvalidValue;
}

MMQ_DEFINE_ERROR_READER(attn_tree)

}  // namespace mmq
