// attn_tree.cu -- attention of a tree's rows over the 8-bit paged cache.
#include "attn_device.cuh"
#include "attn_math.cuh"
#include "internal.h"

namespace mmq {

namespace {

// One warp a row (token and query head): a token at a time, running maximum and sum.
template <int D>
__global__ void __launch_bounds__(128) tree_kernel(const TreeArgs a, int qt, int ot) {
    pdl_wait();
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int t = (int)(row / a.heads), h = (int)(row % a.heads), head = h / a.group;
    if (a.sq.cu && blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.sq.seqs; i += 128)
            if (odd_offsets(a.sq, i, a.sq.cu[i], a.sq.cu[i + 1])) flag_error(DEVERR_LENGTH);
    if (t >= a.sq.tokens) return;
    int s = 0;
    if (a.sq.cu) {
        while (s + 1 < a.sq.seqs && a.sq.cu[s + 1] <= t) s++;
    } else {
        s = t;
    }
    const Seq q = load_seq(a.sq, s, a.c.page);
    if (t < q.n0 || t >= q.n0 + q.n) return;
    const int i = t - q.n0, first = q.len - q.n, end = min(q.end, a.max_kv);
    if (lane == 0 && (q.n > a.max_tokens || end < q.len)) flag_error(DEVERR_LENGTH);
    if (i >= a.max_tokens) return;
    float x[PER], acc[PER];
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const long long at = t * a.q.ts + h * a.q.hs + lane * PER + e;
        x[e] = qt == MMQ_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q.data)[at])
                              : __half2float(static_cast<const __half*>(a.q.data)[at]);
        acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int low = a.window > 0 ? max(first + a.depths[t] - a.window + 1, 0) : 0, blocks = a.c.page / a.c.block;
    for (int j = low; j < end; j++) {
        if (j >= first) {
            const int d = j - first;
            if (d / 32 >= a.words || !(a.masks[(long long)t * a.words + d / 32] >> (d % 32) & 1u)) continue;
        }
        const int pg = a.sq.table[s * a.sq.stride + j / a.c.page], off = j % a.c.page;
        if ((unsigned)pg >= (unsigned long long)a.c.pages) {
            flag_error(DEVERR_PAGE);
            continue;
        }
        const long long ph = (long long)pg * a.c.heads + head, at = (ph * a.c.page + off) * D + lane * PER;
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < PER; e++) dot = fmaf(x[e], (float)a.c.k[at + e], dot);
        const float sc = lane_sum<32>(dot) * a.scale * LOG2E * a.c.ks[ph * blocks + off / a.c.block];
        const float vs = a.c.vs[ph * blocks + off / a.c.block], mn = fmaxf(m, sc), f = ex2(m - mn), p = ex2(sc - mn);
        m = mn;
        l = fmaf(l, f, p);
#pragma unroll
        for (int e = 0; e < PER; e++) acc[e] = fmaf(acc[e], f, p * vs * (float)a.c.v[at + e]);
    }
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const long long at = t * a.out.ts + h * a.out.hs + lane * PER + e;
        const float o = l > 0.f ? acc[e] / l : 0.f;
        if (ot == MMQ_F32) static_cast<float*>(a.out.data)[at] = o;
        else if (ot == MMQ_BF16) static_cast<__nv_bfloat16*>(a.out.data)[at] = __float2bfloat16(o);
        else static_cast<__half*>(a.out.data)[at] = __float2half(o);
    }
    if (lane == 0 && a.lse) a.lse[row] = l > 0.f ? LN2 * (m + log2f(l)) : -INFINITY;
}

}  // namespace

cudaError_t run_attention_tree(int dim, mmq_dtype qt, mmq_dtype ot, const TreeArgs& a, cudaStream_t s) {
    const long long grid = ((long long)a.sq.tokens * a.heads + 3) / 4;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    auto kern = dim == 64 ? tree_kernel<64> : (dim == 128 ? tree_kernel<128> : tree_kernel<256>);
    return launch_pdl(kern, dim3((unsigned)grid), dim3(128), s, a, (int)qt, (int)ot);
}

MMQ_DEFINE_ERROR_READER(attn_tree)

}  // namespace mmq
