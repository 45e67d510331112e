// draft.cu -- the operators around a tree of drafted tokens: what each token sees, and the move of the kept path's rows in
// the 8-bit paged cache.
//
//   masks  sees(i) = {i} + sees(parent(i)),  depth(i) = |sees(i)| - 1
//   keep   place first + kept[i] -> first + i;  s' = max of the scales of a block's tokens, code -> round(code (s/s'))
//
// Both are a few microseconds of dependent loads and little else: masks of 26 tokens 2.8 us, of 256 trees of up to 64 3.2 us (in a
// captured graph); 24 of up to 64 tokens kept in each of 64 sequences, 8 heads of 128, 8.5 us from a cold memory.
#include "attn_device.cuh"
#include "internal.h"

namespace mmq {

namespace {

// ------------------------------------------------------------------------------------------ masks
// One thread block a sequence, one thread a token.  Each round doubles how far a token has looked: it adds what the token
// that its jump leads to sees so far and takes over that one's jump, so a path of d ancestors takes log2 d rounds instead
// of d dependent reads.
__global__ void __launch_bounds__(MMQ_MAX_DRAFT) masks_kernel(const DraftArgs a) {
    pdl_wait();
    extern __shared__ uint32_t s_see[];                       // [tokens][pitch], then two jumps a token
    const int s = blockIdx.x, i = threadIdx.x;
    int n0 = s, n1 = s + 1;
    if (a.cu) {
        n0 = a.cu[s];
        n1 = a.cu[s + 1];
        if (i == 0 && (n1 < n0 || (s == 0 && n0 != 0) || (s == a.seqs - 1 && n1 != a.tokens))) flag_error(DEVERR_LENGTH);
    }
    n0 = max(n0, 0);
    const int asked = max(min(n1, a.tokens) - n0, 0), n = min(asked, a.max_tokens);
    if (i == 0 && asked > n) flag_error(DEVERR_LENGTH);
    if (n == 0) return;
    const int words = (a.max_tokens + 31) / 32, pitch = words | 1, used = (n + 31) / 32;
    int* jumps = reinterpret_cast<int*>(s_see + blockDim.x * pitch);
    uint32_t* mine = s_see + i * pitch;
    int jump = -1;
    if (i < n) {
        jump = a.parents[n0 + i];
        if (jump < -1 || jump >= i) {
            flag_error(DEVERR_DRAFT);
            jump = -1;
        }
    }
    for (int w = 0; w < used; w++) mine[w] = w == i / 32 ? 1u << (i % 32) : 0u;
    for (int round = 0;; round++) {
        int* at = jumps + (round & 1) * blockDim.x;
        at[i] = jump;
        if (!__syncthreads_or(jump >= 0)) break;
        const int from = jump;
        if (from >= 0) jump = at[from];
        for (int w0 = 0; w0 < used; w0 += 4) {                // read, meet, write: four words at a time
            uint32_t v[4] = {};
            if (from >= 0)
#pragma unroll
                for (int w = 0; w < 4; w++)
                    if (w0 + w < used) v[w] = s_see[from * pitch + w0 + w];
            __syncthreads();
            if (from >= 0)
#pragma unroll
                for (int w = 0; w < 4; w++)
                    if (w0 + w < used) mine[w0 + w] |= v[w];
        }
    }
    if (i < n) {
        int seen = 0;
        for (int w = 0; w < used; w++) seen += __popc(mine[w]);
        a.depths[n0 + i] = seen - 1;
    }
    const long long out = (long long)n0 * a.words;
    for (int x = i; x < n * a.words; x += blockDim.x) {
        const int row = x / a.words, w = x - row * a.words;
        a.masks[out + x] = w < used ? s_see[row * pitch + w] : 0u;
    }
}

// ------------------------------------------------------------------------------------------ keep
// One thread block a sequence, head and side (keys or values) goes over the blocks that receive tokens, in their order: a
// token only moves towards the front, so what a block receives lies in it or behind it, and the next block's rows are read
// before this one's are written.  D/16 lanes hold a row.
constexpr int KEEP_THREADS = 128;

template <int D, int B>
__global__ void __launch_bounds__(KEEP_THREADS) keep_kernel(const KeepArgs a) {
    pdl_wait();
    constexpr int LANES = D / 16, ROWS = KEEP_THREADS / LANES, NR = (B + ROWS - 1) / ROWS;
    __shared__ int s_kept[MMQ_MAX_DRAFT];
    __shared__ float s_top[2][KEEP_THREADS / 32];
    const int sh = blockIdx.x / 2, head = sh % a.c.heads, s = sh / a.c.heads;
    const bool isv = blockIdx.x & 1, first = sh == s * a.c.heads && !isv && threadIdx.x == 0;
    const Seq q = load_seq(a.sq, s, a.c.page);
    if (first && a.sq.cu && odd_offsets(a.sq, s, a.sq.cu[s], a.sq.cu[s + 1])) flag_error(DEVERR_LENGTH);
    const int base = q.len - q.n, count = a.counts[s];
    if (base < 0 || q.end < q.len) {
        if (first) flag_error(DEVERR_LENGTH);
        return;
    }
    int bad = count < 0 || count > q.n || count > a.stride, still = 0;
    for (int i0 = 0; !bad && i0 < count; i0 += KEEP_THREADS) {
        const int i = i0 + threadIdx.x;
        int row = i;
        if (i < count) {
            const int32_t* kept = a.kept + s * a.stride + i;
            row = *kept;
            bad = row < 0 || row >= q.n || (i > 0 && row <= kept[-1]);
            s_kept[i] = row;
        }
        bad = __syncthreads_or(bad);
        still += __syncthreads_count(i < count && row == i);  // they come first, as the rows ascend
    }
    if (bad) {
        if (first) flag_error(DEVERR_DRAFT);
        return;
    }
    if (still == count) return;

    const int l = threadIdx.x % LANES, r0 = threadIdx.x / LANES, blocks = a.c.page / B;
    int8_t* codes = isv ? a.c.v : a.c.k;
    float* scales = isv ? a.c.vs : a.c.ks;
    const int32_t* table = a.sq.table + s * a.sq.stride;
    struct Rows {
        uint4 c[NR];
        float scale[NR];
        unsigned live, moved;                                 // bits of the rows
    };
    auto load = [&](int b, Rows& r) {
        r.live = r.moved = 0;
#pragma unroll
        for (int i = 0; i < NR; i++) {
            const int j = r0 + i * ROWS, p = b * B + j;
            r.c[i] = make_uint4(0, 0, 0, 0);
            r.scale[i] = 0.f;
            if (j >= B || p >= base + count) continue;
            const int from = p < base ? p : base + s_kept[p - base];
            r.live |= 1u << i;
            if (from != p) r.moved |= 1u << i;
            const int pg = table[from / a.c.page], off = from % a.c.page;
            if ((unsigned)pg < (unsigned long long)a.c.pages) {
                const long long ph = (long long)pg * a.c.heads + head;
                r.c[i] = *reinterpret_cast<const uint4*>(codes + (ph * a.c.page + off) * D + 16 * l);
                r.scale[i] = scales[ph * blocks + off / B];
            } else if (l == 0) {
                flag_error(DEVERR_PAGE);
            }
        }
    };
    const int b1 = (base + count - 1) / B;
    Rows now, next;
    load((base + still) / B, now);
    for (int b = (base + still) / B; b <= b1; b++) {
        if (b < b1) load(b + 1, next);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NR; i++) top = fmaxf(top, now.scale[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((threadIdx.x & 31) == 0) s_top[b & 1][threadIdx.x >> 5] = top;
        __syncthreads();                                      // also: the block's rows are read
#pragma unroll
        for (int i = 0; i < KEEP_THREADS / 32; i++) top = fmaxf(top, s_top[b & 1][i]);
        const int pg = table[b * B / a.c.page], off = b * B % a.c.page;
        if ((unsigned)pg < (unsigned long long)a.c.pages) {
            const long long ph = (long long)pg * a.c.heads + head;
            int8_t* to = codes + (ph * a.c.page + off) * D + 16 * l;
#pragma unroll
            for (int i = 0; i < NR; i++) {
                const float ratio = top > 0.f ? __fdiv_rn(now.scale[i], top) : 0.f;
                if (!(now.live >> i & 1) || (ratio == 1.f && !(now.moved >> i & 1))) continue;
                uint4 c = now.c[i];
                if (ratio != 1.f) {
                    c.x = scale_codes4(c.x, ratio);
                    c.y = scale_codes4(c.y, ratio);
                    c.z = scale_codes4(c.z, ratio);
                    c.w = scale_codes4(c.w, ratio);
                }
                *reinterpret_cast<uint4*>(to + (long long)(r0 + i * ROWS) * D) = c;
            }
            if (threadIdx.x == 0) scales[ph * blocks + off / B] = top;
        } else if (threadIdx.x == 0) {
            flag_error(DEVERR_PAGE);
        }
        now = next;
    }
}

template <int D>
cudaError_t launch_keep(const KeepArgs& a, cudaStream_t s) {
    const long long grid = 2ll * a.sq.seqs * a.c.heads;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    auto kern = a.c.block == 16 ? keep_kernel<D, 16> : (a.c.block == 32 ? keep_kernel<D, 32> : keep_kernel<D, 64>);
    return launch_pdl(kern, dim3((unsigned)grid), dim3(KEEP_THREADS), s, a);
}

}  // namespace

cudaError_t run_draft_masks(const DraftArgs& a, cudaStream_t s) {
    const int threads = (a.max_tokens + 31) / 32 * 32, words = threads / 32;
    const size_t bytes = (size_t)threads * ((words | 1) + 2) * 4;
    static bool configured[64] = {};
    bool& done = device_flag(configured);
    if (!done) {                                              // as the largest tree takes
        const cudaError_t e = cudaFuncSetAttribute(masks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   MMQ_MAX_DRAFT * (MMQ_MAX_DRAFT / 32 + 3) * 4);
        if (e != cudaSuccess) return e;
        done = true;
    }
    return launch_pdl_smem(masks_kernel, dim3((unsigned)a.seqs), dim3((unsigned)threads), bytes, s, a);
}

cudaError_t run_kv_keep(int dim, const KeepArgs& a, cudaStream_t s) {
    switch (dim) {
        case 64: return launch_keep<64>(a, s);
        case 128: return launch_keep<128>(a, s);
        case 256: return launch_keep<256>(a, s);
    }
    return cudaErrorInvalidValue;
}

MMQ_DEFINE_ERROR_READER(draft)

}  // namespace mmq
