// attn_tree.cu -- attention of a tree's rows over the 8-bit paged cache, on tcgen05.
//
//   t_j = scale log2(e) ks_b (q . k_j) + log2(vs_b),  p_j = 2^(t_j - m),  O = sum_j p_j v_j,  l = sum_b (1/vs_b) sum_{j in b} p_j
//   out = O / l,  lse = ln(2) (m + log2 l)                (the formulas of attn_few.cu) over the j that a row sees
//
// A tree has some ten to a hundred rows (tokens x query heads of a group) for each sequence and key/value head: too many for
// mma.sync, and too few to fill the 128 lanes of a product whose rows they are.  So the products stand the other way round,
// cache tokens and head dimensions on the 128 lanes and the query rows along the columns:
//   S^T [128 tokens x R] = K Q^T       K: fp16 codes in TMEM (A operand), Q: shared memory, K-major
//   O^T [128 dims x R]  += V^T P^T     V: shared memory [token][64 dims of 128 bytes], M-major, P the same way, N-major
// A thread of the softmax then owns a token, with its scales in registers, and R or R/2 rows of it; what it costs goes with the
// rows that there are.  K never passes through shared memory, whose bandwidth is the next bound after the cache's.
//
// One thread block an SM.  The cache tiles of all (sequence, head, row block) units stand in one line, and each block takes an
// equal share of it, wherever that begins and ends (lengths are on the device: the blocks work out the line by themselves);
// units that are cut leave parts in the workspace, which a second launch joins.  Roles:
//   * eight softmax warps in two groups, each half of the rows: a tile's S^T, the mask, the exponentials, P as fp16 to shared
//     memory.  The reference m of a row is raised only when a term passes it by 2^LAZY, which a group votes on; then O is
//     rescaled.  They also bring the queries in and the results out.
//   * four warps turn the codes of K into fp16 in TMEM and four those of V into shared memory, 16 tokens at a time, with several
//     such loads in flight.
//   * one warp issues the products.
#include <algorithm>
#include "attn_device.cuh"
#include "attn_math.cuh"
#include "internal.h"

namespace mmq {

namespace {

constexpr int KT = 128;                      // cache tokens of a tile
constexpr int W_CONVK = 8, W_CONVV = 12, W_MMA = 16;
constexpr int TREE_THREADS = 17 * 32;
constexpr int WINDOW = kChain / KT;          // most tiles that are listed, and summed, in one go
constexpr int SCAN = 512;                    // sequences looked at together
constexpr float UNSET = 1e30f;               // -m of a row that has seen nothing yet

template <int D, int R> struct Tree {
    static constexpr int kChunks = D / 64, kHalves = D == 256 ? 2 : 1;           // 64 dimensions; O^T of 128 dimensions
    static constexpr int kKStages = D == 256 || R == 128 ? 2 : 3;
    static constexpr int kVStages = D == 64 ? 6 : (D == 128 ? 4 : 2);
    static constexpr int kPBufs = D == 128 && R == 128 ? 1 : 2;
    static constexpr int kAhead = D == 64 ? 8 : (D == 128 ? 4 : 2);              // loads of 16 tokens in flight a warp
    static constexpr int kVBytes = KT * D * 2, kQBytes = R * D * 2, kPBytes = KT * R * 2;
    static constexpr int kScaleSlots = 16;
    static constexpr int kKCols = D / 2;
    static constexpr int kOCol = 2 * R, kKCol = kOCol + kHalves * R;
    static_assert(kKCol + kKStages * kKCols <= 512, "TMEM budget");
    // V first: for head_dim 64 the products read the next 16 KB as 64 more dimensions, whose results nothing looks at
    static constexpr int v_off = 0;
    static constexpr int q_off = v_off + kVStages * kVBytes;
    static constexpr int p_off = q_off + kQBytes;
    static constexpr int sc_off = p_off + kPBufs * kPBytes;                      // float4 [slots][8]
    static constexpr int bar_off = sc_off + kScaleSlots * 8 * 16;
    static constexpr int n_bars = 2 * kKStages + 2 * kVStages + kScaleSlots + 6 + 2 + 1;
    static constexpr int misc_off = bar_off + n_bars * 8;
    static constexpr int total = misc_off + 16, alloc = total + 1024;
    static_assert(alloc <= 232448 - 26 * 1024, "shared memory budget (the rest is static)");
};

// A run of tiles of one unit (sequence, key/value head, row block) in the block's share.
struct Piece {
    int s, head, n0;             // n0: first packed row of the sequence
    int first, lim;              // cached tokens before the new ones; tokens past lim do not exist
    int row0, rows;
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
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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
    __device__ uint32_t kfull(int i) const { return b + 8u * i; }
    __device__ uint32_t kempty(int i) const { return b + 8u * (C::kKStages + i); }
    __device__ uint32_t vfull(int i) const { return b + 8u * (2 * C::kKStages + i); }
    __device__ uint32_t vempty(int i) const { return b + 8u * (2 * C::kKStages + C::kVStages + i); }
    __device__ uint32_t scale(int i) const { return b + 8u * (2 * C::kKStages + 2 * C::kVStages + i); }
    __device__ uint32_t rest(int i) const {
        return b + 8u * (2 * C::kKStages + 2 * C::kVStages + C::kScaleSlots + i);
    }
    __device__ uint32_t sfull(int i) const { return rest(i); }                   // S of tiles i mod 2
    __device__ uint32_t pready(int i) const { return rest(2 + i); }
    __device__ uint32_t pvdone(int i) const { return rest(4 + i); }
    __device__ uint32_t qfull() const { return rest(6); }                        // a piece's queries
    __device__ uint32_t ofree() const { return rest(7); }                        // a piece's O is read
    __device__ uint32_t done() const { return rest(8); }
};

// A sequence's place in the line of tiles.
struct Line {
    Seq q;
    int n, base;                 // new tokens, first token of the first tile
    int blocks;                  // row blocks
    long long tiles;             // of a unit
};
template <int R>
__device__ __forceinline__ Line line_of(const TreeArgs& a, int s) {
    Line x;
    x.q = load_seq(a.sq, s, a.c.page);
    x.n = min(x.q.n, a.max_tokens);
    const int first = x.q.len - x.q.n, lim = min(min(x.q.end, a.max_kv), first + x.n);
    x.base = a.window > 0 ? max(first - a.window + 1, 0) / 16 * 16 : 0;
    x.blocks = (x.n * a.group + R - 1) / R;
    x.tiles = max((lim - x.base + KT - 1) / KT, 1);
    return x;
}

template <int D, int R>
__global__ void __launch_bounds__(TREE_THREADS, 1) tree_kernel(const TreeArgs a, const TreeWork work, int qt, int ot) {
    using C = Tree<D, R>;
    constexpr int CH = C::kChunks, NC = R / 64;               // 32-column chunks of a group's rows
    pdl_wait();
    pdl_trigger();                                            // after the wait: the join reads its inputs before its own
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Piece s_piece[WINDOW];
    __shared__ long long s_w[17], s_out[R];
    __shared__ int s_u[17], s_span[2], s_tok[R], s_low[R];
    __shared__ float4 s_col[R / 2];                           // of two rows: factors of S, and -m
    __shared__ float s_m[R], s_fac[R], s_add[R], s_next[R], s_red[2][4][R / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // The line of tiles: every sequence's units one after the other, heads before row blocks.
    const int range = blockIdx.x;
    auto exclusive = [&](long long w, int u, long long& wx, int& ux, long long& wall, int& uall) {
        long long wi = w;
        int ui = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, wi, o);
            const int z = __shfl_up_sync(0xffffffffu, ui, o);
            if (lane >= o) {
                wi += v;
                ui += z;
            }
        }
        __syncthreads();                                      // the arrays' last readers are done
        if (lane == 31) {
            s_w[warp] = wi;
            s_u[warp] = ui;
        }
        __syncthreads();
        wx = wi - w;
        ux = ui - u;
        wall = 0;
        uall = 0;
        for (int i = 0; i < 17; i++) {
            if (i < warp) {
                wx += s_w[i];
                ux += s_u[i];
            }
            wall += s_w[i];
            uall += s_u[i];
        }
    };
    long long all = 0;                                        // tiles of the line
    for (int s0 = 0; s0 < a.sq.seqs; s0 += SCAN) {
        const int s = s0 + threadIdx.x;
        long long w = 0, wx, wall;
        int ux, uall;
        if (threadIdx.x < SCAN && s < a.sq.seqs) {
            const Line x = line_of<R>(a, s);
            w = x.tiles * x.blocks * a.c.heads;
            if (range == 0) {
                const bool odd = a.sq.cu && odd_offsets(a.sq, s, a.sq.cu[s], a.sq.cu[s + 1]);
                if (odd || (x.n > 0 && (x.q.n > x.n || min(x.q.end, a.max_kv) < x.q.len))) flag_error(DEVERR_LENGTH);
            }
        }
        exclusive(w, 0, wx, ux, wall, uall);
        all += wall;
    }
    const long long ranges = min((long long)gridDim.x, all);
    if (range >= ranges) {
        if (threadIdx.x == 0) work.joins[2 * range + 1] = make_int4(0, 0, 0, 0);
        return;                                               // uniform, nothing set up yet
    }
    auto start_of = [&](long long c) { return c * all / ranges; };
    const long long g0 = start_of(range), g1 = start_of(range + 1);

    const uint32_t sb = smem_u32(smem);
    const TreeBars<D, R> bar{sb + C::bar_off};
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc_off + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc_off);
    float4* scales = reinterpret_cast<float4*>(smem + C::sc_off);
    if (warp == W_MMA) {
        if (lane == 0) {
            for (int i = 0; i < C::kKStages; i++) {
                mbar_init(bar.kfull(i), 8);
                mbar_init(bar.kempty(i), 1);
            }
            for (int i = 0; i < C::kVStages; i++) {
                mbar_init(bar.vfull(i), 8);
                mbar_init(bar.vempty(i), 1);
            }
            for (int i = 0; i < C::kScaleSlots; i++) mbar_init(bar.scale(i), 8);
            for (int i = 0; i < 2; i++) {
                mbar_init(bar.sfull(i), 1);
                mbar_init(bar.pready(i), 8);
                mbar_init(bar.pvdone(i), 1);
            }
            mbar_init(bar.qfull(), 8);
            mbar_init(bar.ofree(), 8);
            mbar_init(bar.done(), 1);
            *abort_flag = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    int y0 = 0, k0 = 0;                                       // tiles and pieces of the windows before
    for (long long g = g0; g < g1; g += WINDOW) {
        const long long gz = min(g + WINDOW, g1);
        const int tiles = (int)(gz - g);
        // ---- the window's pieces
        long long wbase = 0;
        int ubase = 0;
        for (int s0 = 0; wbase < gz; s0 += SCAN) {
            const int s = s0 + threadIdx.x;
            long long w = 0, wx, wall;
            int units = 0, ux, uall;
            Line x{};
            if (threadIdx.x < SCAN && s < a.sq.seqs) {
                x = line_of<R>(a, s);
                units = x.blocks * a.c.heads;
                w = x.tiles * units;
            }
            exclusive(w, units, wx, ux, wall, uall);
            wx += wbase;
            ux += ubase;
            if (wx <= g && g < wx + w) s_span[0] = ux + (int)((g - wx) / x.tiles);
            if (wx < gz && gz <= wx + w) s_span[1] = ux + (int)((gz - 1 - wx) / x.tiles);
            __syncthreads();
            if (wx < gz && wx + w > g) {
                const int u0 = s_span[0], first = x.q.len - x.q.n;
                const long long k1 = min((gz - 1 - wx) / x.tiles, (long long)units - 1);
                for (long long k = g > wx ? (g - wx) / x.tiles : 0; k <= k1; k++) {
                    const long long u = wx + k * x.tiles, uz = u + x.tiles, lo = max(u, g), hi = min(uz, gz);
                    Piece p;
                    p.s = s;
                    p.head = (int)(k / x.blocks);
                    p.n0 = x.q.n0;
                    p.first = first;
                    p.lim = min(min(x.q.end, a.max_kv), first + x.n);
                    p.row0 = (int)(k % x.blocks) * R;
                    p.rows = min(x.n * a.group - p.row0, R);
                    p.tok0 = x.base + (int)(lo - u) * KT;
                    p.x0 = (int)(lo - g);
                    p.tiles = (int)(hi - lo);
                    p.slot = 2 * range + (u > g0);
                    p.flags = (lo > max(u, g0) ? P_PREV : 0) | (hi == uz && u >= g0 ? P_DIRECT : 0);
                    s_piece[ux + (int)k - u0] = p;
                    if (g == g0 && u <= g0 && uz > g0) {
                        // the join of the unit that this range begins within, if the range before is the unit's first
                        int parts = 0, slot0 = 0;
                        if (u < g0 && u >= start_of(range - 1)) {
                            parts = (int)((uz * ranges - 1) / all) - (range - 1) + 1;
                            slot0 = 2 * (range - 1) + (u > start_of(range - 1));
                        }
                        work.joins[2 * range] = make_int4(p.n0, p.row0, p.rows, p.head);
                        work.joins[2 * range + 1] = make_int4(parts, slot0, 2 * range, 0);
                    }
                }
            }
            wbase += wall;
            ubase += uall;
        }
        __syncthreads();
        const int pieces = s_span[1] - s_span[0] + 1;

        if (warp >= W_CONVK && warp < W_MMA) {
            // ======================================================= converters
            // Units of 16 tokens (within one page and scale block); warp w of four takes tokens 32w .. of a tile.  Lane (g, t)
            // reads rows g, g+8, 16 bytes at 16t of each 64.
            const bool isv = warp >= W_CONVV;
            const int w = warp & 3, gr = lane >> 2, t = lane & 3, units = 2 * tiles;
            const int blocks = a.c.page / a.c.block;
            const int8_t* codes = (isv ? a.c.v : a.c.k) + gr * D + 16 * t;
            long long src = -1;                               // lane i: the i-th of the warp's next 32 units (negative: zeros)
            float ks = 0.f, lv = -INFINITY, iv = 0.f;
            auto lookup = [&](int v0) {
                const int v = v0 + lane, x = v >> 1;
                src = -1, ks = 0.f, lv = -INFINITY, iv = 0.f;
                if (v >= units) return;
                int lo = 0, hi = pieces;                      // the piece that tile x lies in
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (s_piece[mid].x0 <= x) lo = mid;
                    else hi = mid;
                }
                const Piece& p = s_piece[lo];
                const int tok = p.tok0 + (x - p.x0) * KT + 32 * w + 16 * (v & 1);
                if (tok >= p.lim) return;
                const int page = tok / a.c.page, off = tok - page * a.c.page;
                const int pg = a.sq.table[p.s * a.sq.stride + page];
                if ((unsigned)pg < (unsigned long long)a.c.pages) {
                    const long long ph = (long long)pg * a.c.heads + p.head;
                    src = (ph * a.c.page + off) * D;
                    if (!isv) {
                        const long long sc = ph * blocks + off / a.c.block;
                        ks = a.c.ks[sc];
                        const float vs = fmaxf(a.c.vs[sc], SCALE_FLOOR);
                        lv = __log2f(vs);
                        iv = __fdividef(1.f, vs);
                    }
                } else {
                    flag_error(DEVERR_PAGE);
                }
            };
            uint4 r[C::kAhead][2][CH];
            auto load = [&](int v, uint4 (&to)[2][CH]) {
                if (v >= units) return;
                if ((v & 31) == 0) lookup(v);
                const long long at = __shfl_sync(0xffffffffu, src, v & 31);
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int c = 0; c < CH; c++)
                        to[h][c] = at >= 0 ? ld_cache(codes + at + 8 * h * D + 64 * c) : make_uint4(0, 0, 0, 0);
                // (the slot's last readers are far behind: K runs at most kKStages + 1 tiles ahead of the softmax, these
                // loads kAhead / 2 more)
                if (!isv && lane == (v & 31))
                    scales[(y0 + (v >> 1)) % C::kScaleSlots * 8 + 2 * w + (v & 1)] = make_float4(ks, lv, iv, 0.f);
            };
            static_assert(C::kKStages + 2 + C::kAhead / 2 < C::kScaleSlots, "scale slots");
            bool ok = true;
#pragma unroll
            for (int i = 0; i < C::kAhead; i++) load(i, r[i]);
            for (int v0 = 0; ok && v0 < units; v0 += C::kAhead) {
#pragma unroll
                for (int i = 0; i < C::kAhead; i++) {
                    const int v = v0 + i, y = y0 + (v >> 1);
                    if (v >= units || !ok) continue;
                    if (isv) {
                        const int st = y % C::kVStages;
                        ok = mbar_wait(bar.vempty(st), ((y / C::kVStages) & 1) ^ 1, abort_flag);
                        if (!ok) continue;
                        const uint32_t to = sb + C::v_off + st * C::kVBytes;
#pragma unroll
                        for (int h = 0; h < 2; h++)
#pragma unroll
                            for (int c = 0; c < CH; c++) {
                                const uint4 x = r[i][h][c];
                                uint32_t z[8];
                                codes_even_odd(x.x, z[0], z[1]);
                                codes_even_odd(x.y, z[2], z[3]);
                                codes_even_odd(x.z, z[4], z[5]);
                                codes_even_odd(x.w, z[6], z[7]);
                                const uint32_t at = to + c * (KT * 128), row = 32 * w + 16 * (v & 1) + 8 * h + gr;
                                st_shared_v4(at + sw128_off(row, 2 * t), z[0], z[1], z[2], z[3]);
                                st_shared_v4(at + sw128_off(row, 2 * t + 1), z[4], z[5], z[6], z[7]);
                            }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar.vfull(st));
                    } else {
                        const int st = y % C::kKStages;
                        ok = mbar_wait(bar.kempty(st), ((y / C::kKStages) & 1) ^ 1, abort_flag);
                        if (!ok) continue;
                        tc_fence_after();
                        const uint32_t to = tmem + ((uint32_t)(32 * w + 16 * (v & 1)) << 16) + C::kKCol + st * C::kKCols;
#pragma unroll
                        for (int c = 0; c < CH; c++) {
                            uint32_t z[16];
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const uint4 x = r[i][h][c];
                                codes_even_odd(x.x, z[2 * h], z[2 * h + 1]);
                                codes_even_odd(x.y, z[4 + 2 * h], z[4 + 2 * h + 1]);
                                codes_even_odd(x.z, z[8 + 2 * h], z[8 + 2 * h + 1]);
                                codes_even_odd(x.w, z[12 + 2 * h], z[12 + 2 * h + 1]);
                            }
                            tmem_st_16x256b_x4(to + 32 * c, z);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar.kfull(st));
                            mbar_arrive(bar.scale(y % C::kScaleSlots));
                        }
                    }
                    load(v + C::kAhead, r[i]);
                }
            }
        } else if (warp == W_MMA) {
            // ======================================================= products
            constexpr uint32_t idesc_s = idesc_f16_f32(128, R);
            constexpr uint32_t idesc_o = idesc_f16_f32(128, R) | (1u << 15) | (1u << 16);     // M and N along the rows
            const uint32_t q_lo = desc_lo(sb + C::q_off, 16), v_lo = desc_lo(sb + C::v_off, KT * 128);
            const uint32_t p_lo = desc_lo(sb + C::p_off, KT * 128);
            bool ok = true;
            int ks = 0, kx = s_piece[0].x0;                   // the piece whose S comes next, and its first tile
            auto product_s = [&](int x) {
                const int y = y0 + x, st = y % C::kKStages;
                if (x == kx) {
                    ok = ok && mbar_wait(bar.qfull(), (k0 + ks) & 1, abort_flag);
                    ks++;
                    kx = ks < pieces ? s_piece[ks].x0 : tiles;
                }
                ok = ok && mbar_wait(bar.kfull(st), (y / C::kKStages) & 1, abort_flag);
                if (!ok) return;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; k++)
                        umma_ts(tmem + (y & 1) * R, tmem + C::kKCol + st * C::kKCols + 8 * k,
                                q_lo + (k / 4) * (R * 128 >> 4) + 2 * (k % 4), idesc_s, k > 0);
                    umma_commit(bar.sfull(y & 1));
                    umma_commit(bar.kempty(st));
                }
                __syncwarp();
            };
            product_s(0);
            int ko = 0;                                       // the piece whose O is summed
            for (int x = 0; ok && x < tiles; x++) {
                const int y = y0 + x, st = y % C::kVStages;
                while (x >= s_piece[ko].x0 + s_piece[ko].tiles) ko++;
                const bool fresh = x == s_piece[ko].x0, more = x + 1 < tiles, ahead = more && x + 1 != kx;
                if (ahead) product_s(x + 1);
                ok = ok && mbar_wait(bar.vfull(st), (y / C::kVStages) & 1, abort_flag);
                if (fresh && k0 + ko > 0) ok = ok && mbar_wait(bar.ofree(), (k0 + ko - 1) & 1, abort_flag);
                ok = ok && mbar_wait(bar.pready(y & 1), (y >> 1) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t p = p_lo + (y % C::kPBufs) * (C::kPBytes >> 4), v = v_lo + st * (C::kVBytes >> 4);
#pragma unroll
                    for (int h = 0; h < C::kHalves; h++)
#pragma unroll
                        for (int k = 0; k < KT / 16; k++)
                            umma_ss(tmem + C::kOCol + h * R, v + h * (2 * KT * 128 >> 4) + k * (2048 >> 4),
                                    p + k * (2048 >> 4), idesc_o, !fresh || k > 0);
                    umma_commit(bar.pvdone(y & 1));
                    umma_commit(bar.vempty(st));
                }
                __syncwarp();
                if (more && !ahead) product_s(x + 1);
            }
        } else {
            // ======================================================= softmax: one thread a token
            // A failed wait does not leave the loops (the group meets at barriers); later waits then return at once.
            const int grp = warp >> 2, w = warp & 3, tk = 32 * w + lane, gt = threadIdx.x & 127, c0 = grp * (R / 2);
            const int id = 1 + grp;
            constexpr int LPR = D / 8, RPP = 4 * 32 / LPR;    // lanes on a row of queries, rows at a time
            const uint32_t lanes = (uint32_t)(32 * w) << 16;
            bool ok = true;
            auto fetch_q = [&](const Piece& p) {
                if (p.rows <= c0) return;
#pragma unroll
                for (int i = 0; i < R / 2; i += RPP) {
                    const int c = c0 + i + (w * 32 + lane) / LPR, row = p.row0 + min(c, p.rows - 1), m = lane % LPR;
                    const uint16_t* from = static_cast<const uint16_t*>(a.q.data) + (long long)(p.n0 + row / a.group) * a.q.ts +
                                           (long long)(p.head * a.group + row % a.group) * a.q.hs + 8 * m;
                    cp_async_16(sb + C::q_off + (m / 8) * (R * 128) + sw128_off(c, m % 8), from, c < p.rows ? 16 : 0);
                }
                cp_async_commit();
            };
            // In place to fp16, each row times the power of two that brings its largest magnitude to [1, 2), in the order in
            // which K's dimensions stand: group w of four dimensions of 16t .. 16t + 15 at place 4w + t, 0 2 1 3 within.
            auto convert_q = [&](const Piece& p) {
                if (p.rows > c0) {
                    cp_async_wait<0>();
#pragma unroll 2
                    for (int i = 0; i < R / 2; i += RPP) {
                        const int c = c0 + i + (w * 32 + lane) / LPR, m = lane % LPR;
                        const uint32_t panel = sb + C::q_off + (m / 8) * (R * 128);
                        float x[8], top = 0.f, up, down;
                        unpack8(ld_shared_u4(panel + sw128_off(c, m % 8)), qt == MMQ_BF16, x);
#pragma unroll
                        for (int e = 0; e < 8; e++) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
                        for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        row_scale(top, up, down);
                        __syncwarp();                         // the rows are read
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int four = 2 * (m % 8) + e, place = 4 * (four & 3) + (four >> 2);
                            const uint32_t lo = pack2(x[4 * e] * up, x[4 * e + 2] * up, __half());
                            const uint32_t hi = pack2(x[4 * e + 1] * up, x[4 * e + 3] * up, __half());
                            asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(panel + sw128_off(c, place >> 1) + 8 * (place & 1)),
                                         "r"(lo), "r"(hi)
                                         : "memory");
                        }
                        if (m == 0) s_next[c] = a.scale * LOG2E * down;
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.qfull());
            };
            fetch_q(s_piece[0]);
            convert_q(s_piece[0]);
            for (int k = 0; k < pieces; k++) {
                const Piece p = s_piece[k];
                const bool busy = p.rows > c0, more = k + 1 < pieces;
                named_bar_sync(id, 128);                      // s_next is there, the last piece's values are read
                if (gt < R / 2) {
                    const int c = c0 + gt, row = p.row0 + min(c, p.rows - 1), tok = p.n0 + row / a.group;
                    const bool real = c < p.rows;
                    float* col = reinterpret_cast<float*>(&s_col[c / 2]) + (c & 1);
                    col[0] = real ? s_next[c] : 0.f;
                    col[2] = real ? UNSET : -INFINITY;
                    s_m[c] = -INFINITY;
                    s_tok[c] = tok;
                    if (a.window > 0) s_low[c] = p.first + a.depths[tok] - a.window + 1;
                    s_out[c] = (long long)tok * a.out.ts + (p.head * a.group + row % a.group) * a.out.hs;
                }
                named_bar_sync(id, 128);
                uint64_t l2[NC][16];
#pragma unroll
                for (int h = 0; h < NC; h++)
#pragma unroll
                    for (int i = 0; i < 16; i++) l2[h][i] = 0ull;
                for (int x = p.x0; x < p.x0 + p.tiles; x++) {
                    const int y = y0 + x, tok = p.tok0 + (x - p.x0) * KT, j = tok + tk;
                    // which rows see the token: all, but for the new tokens and the window's edge
                    const bool masked = tok + KT > p.first || (a.window > 0 && tok <= p.first + a.max_tokens - a.window);
                    uint32_t see[NC];
#pragma unroll
                    for (int h = 0; h < NC; h++) see[h] = 0xFFFFFFFFu;
                    if (masked && busy) {
                        const int d = j - p.first;
#pragma unroll
                        for (int h = 0; h < NC; h++) {
                            if (j >= p.lim) {
                                see[h] = 0u;
                            } else if (d >= 0) {
                                uint32_t bits = 0u;
                                if (d / 32 < a.words)
#pragma unroll 8
                                    for (int i = 0; i < 32; i++)
                                        bits |= (a.masks[(long long)s_tok[c0 + 32 * h + i] * a.words + d / 32] >> (d % 32) & 1u)
                                                << i;
                                see[h] = bits;
                            } else if (a.window > 0) {
#pragma unroll 8
                                for (int i = 0; i < 32; i++)
                                    if (j < s_low[c0 + 32 * h + i]) see[h] &= ~(1u << i);
                            }
                        }
                    }
                    ok = mbar_wait(bar.scale(y % C::kScaleSlots), (y / C::kScaleSlots) & 1, abort_flag) && ok;
                    ok = mbar_wait(bar.sfull(y & 1), (y >> 1) & 1, abort_flag) && ok;
                    tc_fence_after();
                    if (more && x + 1 == p.x0 + p.tiles) fetch_q(s_piece[k + 1]);             // every S of the piece is complete
                    if (busy) {
                        const float4 sc = scales[y % C::kScaleSlots * 8 + tk / 16];
                        const uint64_t ks2 = f2_pack(sc.x, sc.x), lv2 = f2_pack(sc.y, sc.y), iv2 = f2_pack(sc.z, sc.z);
#pragma unroll
                        for (int h = 0; h < NC; h++) {
                            const int cb = c0 + 32 * h;
                            uint32_t xr[32];
                            float e[32];
                            auto terms = [&](bool shifted) {  // e = t - m, or t
                                tmem_ld32(tmem + lanes + (y & 1) * R + cb, xr);
                                tmem_wait32(xr);
#pragma unroll
                                for (int i = 0; i < 16; i++) {
                                    const float4 f = s_col[cb / 2 + i];
                                    const uint64_t sh = shifted ? f2_add(f2_pack(f.z, f.w), lv2) : lv2;
                                    const uint64_t s2 = f2_pack(__uint_as_float(xr[2 * i]), __uint_as_float(xr[2 * i + 1]));
                                    f2_unpack(f2_fma(s2, f2_mul(f2_pack(f.x, f.y), ks2), sh), e[2 * i], e[2 * i + 1]);
                                }
                                if (masked)
#pragma unroll
                                    for (int i = 0; i < 32; i++)
                                        if (!(see[h] >> i & 1u)) e[i] = -INFINITY;
                            };
                            terms(true);
                            float top = e[31];
#pragma unroll
                            for (int i = 0; i < 30; i += 2) top = max3(top, e[i], e[i + 1]);
                            top = fmaxf(top, e[30]);
                            if (group_any(id, top > LAZY)) {
                                terms(false);
                                const float mine = across<true>(e);
                                s_red[grp][w][32 * h + lane] = mine;
                                named_bar_sync(id, 128);
                                if (gt < 32) {
                                    const int c = cb + gt;
                                    const float(&red)[4][R / 2] = s_red[grp];
                                    const int at = 32 * h + gt;
                                    const float most = fmaxf(fmaxf(red[0][at], red[1][at]), fmaxf(red[2][at], red[3][at]));
                                    const float m = s_m[c], mn = fmaxf(m, most - HEAD);
                                    s_fac[c] = m == -INFINITY ? 1.f : ex2(m - mn);
                                    if (c < p.rows && mn > -INFINITY) {
                                        s_m[c] = mn;
                                        reinterpret_cast<float*>(&s_col[c / 2])[2 + (c & 1)] = -mn;
                                    }
                                }
                                named_bar_sync(id, 128);
                                uint64_t fac[16];
#pragma unroll
                                for (int i = 0; i < 16; i++) {
                                    fac[i] = f2_pack(s_fac[cb + 2 * i], s_fac[cb + 2 * i + 1]);
                                    l2[h][i] = f2_mul(l2[h][i], fac[i]);
                                }
                                if (x > p.x0) {
                                    ok = mbar_wait(bar.pvdone((y - 1) & 1), ((y - 1) >> 1) & 1, abort_flag) && ok;
                                    tc_fence_after();
#pragma unroll
                                    for (int o = 0; o < C::kHalves; o++) {
                                        const uint32_t at = tmem + lanes + C::kOCol + o * R + cb;
                                        tmem_ld32(at, xr);
                                        tmem_wait32(xr);
#pragma unroll
                                        for (int i = 0; i < 16; i++) {
                                            float z0, z1;
                                            f2_unpack(f2_mul(f2_pack(__uint_as_float(xr[2 * i]), __uint_as_float(xr[2 * i + 1])),
                                                             fac[i]), z0, z1);
                                            xr[2 * i] = __float_as_uint(z0);
                                            xr[2 * i + 1] = __float_as_uint(z1);
                                        }
                                        tmem_st32(at, xr);
                                    }
                                    tmem_st_wait();
                                }
                                terms(true);
                            }
                            // P's buffer is free once the product that read it is complete
                            if (h == 0 && y >= C::kPBufs)
                                ok = mbar_wait(bar.pvdone((y - C::kPBufs) & 1), ((y - C::kPBufs) >> 1) & 1, abort_flag) && ok;
                            const uint32_t row = sb + C::p_off + (y % C::kPBufs) * C::kPBytes + (cb / 64) * (KT * 128);
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                uint32_t z[4];
#pragma unroll
                                for (int u = 0; u < 4; u++) {
                                    const float p0 = ex2(e[8 * i + 2 * u]), p1 = ex2(e[8 * i + 2 * u + 1]);
                                    l2[h][4 * i + u] = f2_fma(f2_pack(p0, p1), iv2, l2[h][4 * i + u]);
                                    z[u] = pack2(p0, p1, __half());
                                }
                                st_shared_v4(row + sw128_off(tk, cb % 64 / 8 + i), z[0], z[1], z[2], z[3]);
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar.pready(y & 1));
                }
                if (more) convert_q(s_piece[k + 1]);
                // ---- the piece's result
                const int yz = y0 + p.x0 + p.tiles - 1;
                ok = mbar_wait(bar.pvdone(yz & 1), (yz >> 1) & 1, abort_flag) && ok;
                tc_fence_after();
                if (busy) {
#pragma unroll
                    for (int h = 0; h < NC; h++) {
                        float e[32];
#pragma unroll
                        for (int i = 0; i < 16; i++) f2_unpack(l2[h][i], e[2 * i], e[2 * i + 1]);
                        s_red[grp][w][32 * h + lane] = across<false>(e);
                    }
                    named_bar_sync(id, 128);
                    if (gt < R / 2 && c0 + gt < p.rows) {
                        const int c = c0 + gt;
                        const float(&red)[4][R / 2] = s_red[grp];
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
                            const int row = p.row0 + c;
                            if (ok && a.lse)
                                a.lse[(long long)s_tok[c] * a.heads + p.head * a.group + row % a.group] =
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
                        for (int b = 0; b < NC * C::kHalves; b++) {
                            const int o = b / NC, cb = c0 + 32 * (b % NC), d = 128 * o + dim;
                            if (cb >= p.rows) continue;
                            uint32_t xr[32];
                            tmem_ld32(tmem + lanes + C::kOCol + o * R + cb, xr);
                            tmem_wait32(xr);
                            float* part = work.part_o + ((long long)p.slot * R + cb) * D + d;
#pragma unroll
                            for (int i = 0; i < 32; i++) {
                                if (cb + i >= p.rows) break;
                                const float keep = s_fac[cb + i];
                                float v = keep == 0.f ? 0.f : __uint_as_float(xr[i]) * keep;
                                if (p.flags & P_PREV) v = fmaf(part[i * D], s_add[cb + i], v);
                                if (p.flags & P_DIRECT) {
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
        }
        __syncthreads();                                      // every role is done with the window
        y0 += tiles;
        k0 += pieces;
        if (*abort_flag) break;                               // (nothing waits here: the same for all)
    }
    if (warp == W_MMA) {
        if (elect_one()) umma_commit(bar.done());
        __syncwarp();
        mbar_wait_final(bar.done(), 0);
        __syncwarp();
    }
    // ---- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
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
    const int4 unit = work.joins[2 * c];                      // first packed row, row block, rows, head
    if (row >= unit.z) return;
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
    const int r = unit.y + row, h = unit.w * a.group + r % a.group;
    const long long tok = unit.x + r / a.group, at = tok * a.out.ts + h * a.out.hs + lane;
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
    cudaError_t e = launch_pdl_smem(kern, dim3((unsigned)p.ranges), dim3(TREE_THREADS), Tree<D, R>::alloc, s, a, work, (int)qt,
                                    (int)ot);
    if (e != cudaSuccess || p.ranges == 1) return e;
    if (p.many_parts)
        return launch_pdl(tree_join_kernel<D, 4>, dim3((unsigned)((p.ranges - 1) * R)), dim3(128), s, a, work, R, (int)ot);
    return launch_pdl(tree_join_kernel<D, 1>, dim3((unsigned)((p.ranges - 1) * (R / 4))), dim3(128), s, a, work, R, (int)ot);
}

}  // namespace

// Shares of the line of tiles: one a multiprocessor, but none below two tiles of what the bounds allow (a block's start
// and the join cost more).
TreePlan tree_plan(long long tokens, int heads, int kv_heads, int dim, int seqs, long long max_tokens, long long max_kv) {
    constexpr long long SMS = 152, LEAST = 2;
    TreePlan p{};
    const long long group = heads / kv_heads, rows = max_tokens * group;
    p.rows = dim == 256 || rows <= 64 ? 64 : 128;
    const long long each = seqs * ((rows + p.rows - 1) / p.rows), packed = tokens * group / p.rows + seqs;
    const long long units = kv_heads * std::min(each, packed), tiles = std::max((max_kv + KT - 1) / KT, 1ll);
    const long long shares = (units * tiles + LEAST - 1) / LEAST;
    p.ranges = (int)std::min(shares, SMS);
    p.many_parts = units <= SMS / 8;
    size_t off = 0;
    p.joins = off;
    off += ((size_t)p.ranges * 2 * sizeof(int4) + 255) & ~size_t(255);
    p.part_ml = off;
    off += ((size_t)p.ranges * 2 * p.rows * sizeof(float2) + 255) & ~size_t(255);
    p.part_o = off;
    off += (size_t)p.ranges * 2 * p.rows * dim * sizeof(float);
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
