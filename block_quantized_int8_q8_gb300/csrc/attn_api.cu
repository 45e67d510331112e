// attn_api.cu -- the extern "C" boundary of the attention operators (declared and documented in include/mmq.h):
// argument checks, workspace layout, launches on the caller's stream.
#include <cmath>
#include "attn.h"
#include "internal.h"

using namespace mmq;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int type_size(mmq_dtype t) { return t == MMQ_F32 ? 4 : 2; }
bool known_dtype(mmq_dtype t) { return t == MMQ_F32 || t == MMQ_BF16 || t == MMQ_F16; }

mmq_status check_rows(const mmq_heads* r) {
    if (!r || !r->data || !known_dtype(r->dtype)) return MMQ_ERR_INVALID_ARG;
    if (r->token_stride < 0 || r->head_stride < 0) return MMQ_ERR_INVALID_ARG;
    const int per = 16 / type_size(r->dtype);
    if (!aligned16(r->data) || r->token_stride % per || r->head_stride % per) return MMQ_ERR_ALIGN;
    return MMQ_OK;
}
HeadRows rows_of(const mmq_heads* r) { return r ? HeadRows{r->data, r->token_stride, r->head_stride} : HeadRows{}; }

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

mmq_status check_weight(const float* w) { return aligned16(w) ? MMQ_OK : MMQ_ERR_ALIGN; }

mmq_status check_rotary(const mmq_rotary* r, int dim) {
    if (!r) return MMQ_OK;
    if (r->rot_dim <= 0 || r->rot_dim % 8 || r->rot_dim > dim || r->positions <= 0) return MMQ_ERR_SHAPE;
    if (!r->cos || !r->sin) return MMQ_ERR_INVALID_ARG;
    return aligned16(r->cos) && aligned16(r->sin) ? MMQ_OK : MMQ_ERR_ALIGN;
}
RotaryArgs rotary_of(const mmq_rotary* r) {
    return r ? RotaryArgs{r->cos, r->sin, r->positions, r->rot_dim / 2, r->interleaved != 0} : RotaryArgs{};
}

mmq_status check_cache(const mmq_kv_cache* c) {
    if (!c) return MMQ_ERR_INVALID_ARG;
    if (!head_dim_ok(c->head_dim) || c->kv_heads <= 0 || c->pages <= 0) return MMQ_ERR_SHAPE;
    if (c->block != 16 && c->block != 32 && c->block != 64) return MMQ_ERR_SHAPE;
    if (c->page_size <= 0 || c->page_size > 32768 || c->page_size % c->block) return MMQ_ERR_SHAPE;
    if (c->pages > kMaxDim || c->pages * c->kv_heads > kMaxDim) return MMQ_ERR_SHAPE;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return MMQ_ERR_INVALID_ARG;
    return aligned16(c->k) && aligned16(c->v) && aligned16(c->k_scale) && aligned16(c->v_scale) ? MMQ_OK
                                                                                               : MMQ_ERR_ALIGN;
}
CacheArgs cache_of(const mmq_kv_cache* c) {
    return CacheArgs{c->k, c->v, c->k_scale, c->v_scale, c->pages, c->kv_heads, c->page_size, c->block};
}

// MMQ_OK with *work = false where there is nothing to do.
mmq_status check_seqs(const mmq_kv_seqs* q, int64_t tokens, bool* work) {
    *work = false;
    if (!q || q->seqs < 0 || tokens < 0) return MMQ_ERR_INVALID_ARG;
    if (tokens > kMaxDim) return MMQ_ERR_SHAPE;
    if (!q->cu_tokens && tokens != q->seqs) return MMQ_ERR_INVALID_ARG;
    if (tokens == 0 || q->seqs == 0) return tokens == 0 ? MMQ_OK : MMQ_ERR_INVALID_ARG;
    if (q->table_stride <= 0 || q->table_stride > kMaxDim) return MMQ_ERR_SHAPE;
    if (!q->page_table || !q->kv_lens) return MMQ_ERR_INVALID_ARG;
    if (!aligned16(q->page_table) || !aligned16(q->kv_lens) || !aligned16(q->cu_tokens)) return MMQ_ERR_ALIGN;
    *work = true;
    return MMQ_OK;
}
SeqArgs seqs_of(const mmq_kv_seqs* q, int64_t tokens) {
    return SeqArgs{q->page_table, q->table_stride, q->kv_lens, q->cu_tokens, q->seqs, (int)tokens};
}

cudaStream_t stream_of(mmq_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

mmq_status done(cudaError_t e, const char* where) { return e == cudaSuccess ? MMQ_OK : record_cuda_failure(e, where); }

#define MMQ_TRY(expr)                                  \
    do {                                               \
        const mmq_status st_ = (expr);                 \
        if (st_ != MMQ_OK) return st_;                 \
    } while (0)

// What mmq_kv_append and mmq_kv_append_tree (tree given) share.
mmq_status append(const mmq_kv_cache* cache, const mmq_kv_seqs* seqs, const mmq_draft_tree* tree, int64_t tokens,
                  const mmq_heads* k, const mmq_heads* v, const float* k_weight, const mmq_heads* q, int q_heads,
                  const float* q_weight, const mmq_heads* q_out, const mmq_rotary* rotary, float eps, cudaStream_t s,
                  const char* where) {
    MMQ_TRY(check_cache(cache));
    bool work;
    MMQ_TRY(check_seqs(seqs, tokens, &work));
    MMQ_TRY(check_rotary(rotary, cache->head_dim));
    if (!q != !q_out || (q && q_heads <= 0)) return MMQ_ERR_INVALID_ARG;
    if (!work) return MMQ_OK;
    if (tree && !tree->depths) return MMQ_ERR_INVALID_ARG;
    if (tree && !aligned16(tree->depths)) return MMQ_ERR_ALIGN;
    MMQ_TRY(check_rows(k));
    MMQ_TRY(check_rows(v));
    if (q) MMQ_TRY(check_rows(q));
    if (q) MMQ_TRY(check_rows(q_out));
    if (k->dtype != v->dtype || (q && q->dtype != k->dtype)) return MMQ_ERR_UNSUPPORTED;
    MMQ_TRY(check_weight(k_weight));
    MMQ_TRY(check_weight(q_weight));
    AppendArgs a{};
    a.c = cache_of(cache);
    a.sq = seqs_of(seqs, tokens);
    a.k = rows_of(k);
    a.v = rows_of(v);
    a.q = rows_of(q);
    a.q_out = rows_of(q_out);
    a.k_weight = k_weight;
    a.q_weight = q ? q_weight : nullptr;
    a.q_heads = q ? q_heads : 0;
    a.rot = rotary_of(rotary);
    a.eps = eps;
    a.depths = tree ? tree->depths : nullptr;
    return done(run_kv_append(cache->head_dim, k->dtype, q ? q_out->dtype : k->dtype, a, s), where);
}

}  // namespace

namespace mmq {

// Few rows (new tokens x query heads of a key/value head <= 16) run on the few-row kernel, more on the tiled one.
// The cache range is cut in chunks where the row blocks alone would not fill the GPU.
//   few rows: all thread blocks do equal work on equal lengths, so the chunks are cut to make one wave; ragged
//     lengths even out from 2048 tokens down.  Several sequences whose pairs with a head fill less than half of a wave
//     leave a second wave nearly empty at that size and take 1024 (heads of 128, 8 key/value heads, ragged: 8 and 16
//     sequences of up to 20 k tokens 48.5 -> 44.6 and 74.8 -> 68.5 us).  More pairs make many waves anyway, and smaller
//     parts only add starts and joins (200 of up to 2000 tokens: 78 -> 83 us; 64 of up to 8192 at head_dim 64 and 256:
//     59 -> 62 and 183 -> 195).
//   tiled: one thread block fits on an SM, and its start and end cost about as much as five tiles.  B < 152 of them leave
//     SMs idle, so every range of T tokens is cut at c = B (T + 640) / 152: the B whole parts take an SM each, and the
//     last, shorter ones go one after the other to the SMs left over, all done at about the same time.  (128 blocks of
//     32 k tokens: 425 us whole, 455 us in two equal parts, 464 us in seven.)  No cut for a rest below ten tiles.
//     A part of more than kChain tokens needs its rows' places in the workspace even where it is the only one.
// A window shortens the range that a sequence's rows see together; the parts stay within what max_kv alone would give,
// so that the workspace does not depend on it.  One that no sequence outgrows hides nothing and is none: the largest
// values of its type, a common way to ask for none, take no part in any sum.
AttnPlan attention_plan(long long tokens, int heads, int kv_heads, int dim, int seqs, long long max_tokens,
                        long long max_kv, long long window) {
    return attention_plan_of(max_tokens * (heads / kv_heads) <= kFewRows, tokens, heads, kv_heads, dim, seqs, max_tokens, max_kv,
                             window);
}

AttnPlan attention_plan_of(bool few, long long tokens, int heads, int kv_heads, int dim, int seqs, long long max_tokens,
                           long long max_kv, long long window) {
    AttnPlan p{};
    constexpr long long SMS = 152;
    const long long rows = max_tokens * (heads / kv_heads);
    p.few = few;
    const long long pairs = (long long)seqs * kv_heads * (p.few ? (rows + kFewRows - 1) / kFewRows : 1), granule = p.few ? 64 : 128;
    auto cut = [&](long long range) {                         // tokens of a part
        if (p.few) {
            const long long slots = few_blocks(dim, rows <= 8 ? 1 : 2) * SMS, want = (slots + pairs - 1) / pairs;
            const long long chunk = ((range + want - 1) / want + granule - 1) / granule * granule;
            const long long most = seqs > 1 && 2 * pairs <= slots ? 1024 : 2048;
            return chunk < 128 ? 128ll : (chunk > most ? most : chunk);
        }
        const long long block = dim == 256 ? 128 : 256, group = heads / kv_heads;
        const long long packed = tokens * group / block + seqs, each = seqs * ((rows + block - 1) / block);
        const long long blocks = kv_heads * (packed < each ? packed : each);
        const long long whole = (range + granule - 1) / granule * granule;
        const long long chunk = blocks < SMS ? (blocks * (range + 640) / SMS + granule - 1) / granule * granule : whole;
        return chunk + 1280 > range ? (whole > 512 ? whole : 512ll) : (chunk < 512 ? 512ll : chunk);
    };
    auto parts = [](long long range, long long chunk) { return range > chunk ? (range + chunk - 1) / chunk : 1; };
    long long chunk = cut(max_kv);
    const long long most = parts(max_kv, chunk);
    p.splits = (int)most;
    p.window = window < max_kv ? (int)window : 0;
    const long long seen = max_tokens + p.window + 30;        // in whole tiles of 16
    if (p.window > 0 && seen < max_kv) {
        chunk = cut(seen);
        while (parts(seen, chunk) > most) chunk += granule;
        p.splits = (int)parts(seen, chunk);
    }
    p.chunk = (int)chunk;
    size_t off = 0;
    if (p.splits > 1 || (!p.few && chunk > kChain)) {
        const size_t all = (size_t)tokens * heads * p.splits;
        p.part_ml = off;
        off += (all * sizeof(float2) + 255) & ~size_t(255);
        p.part_o = off;
        off += (all * dim * sizeof(float) + 255) & ~size_t(255);
    }
    p.total = off;
    return p;
}

namespace {

AttnArgs attention_args(const mmq_heads* q, int n_heads, const mmq_kv_cache* cache, const mmq_kv_seqs* seqs, int64_t tokens,
                        int64_t max_tokens, int64_t max_kv_len, float scale, int causal, const AttnPlan& p,
                        const mmq_heads* out, float* lse, void* workspace) {
    AttnArgs a{};
    a.q = rows_of(q);
    a.out = rows_of(out);
    a.c = cache_of(cache);
    a.sq = seqs_of(seqs, tokens);
    a.heads = n_heads;
    a.group = n_heads / cache->kv_heads;
    a.max_tokens = (int)max_tokens;
    a.max_kv = (int)max_kv_len;
    a.scale = scale;
    a.causal = causal != 0;
    a.window = p.window;
    a.lse = lse;
    if (p.total > 0) {
        a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.part_ml);
        a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.part_o);
    }
    return a;
}

}  // namespace

// Which kernel a tree's rows take.  Microseconds below: a captured call from a cold L2, 32 query and 8 key/value heads of 128
// unless stated, bounds that hold; "one of 2000" is one sequence of 2000 cached tokens.
// FEW, the few-row kernel: for 16 rows (32 of head_dim 64), of which tiles of 64 would leave most empty, and for small problems,
//   whose blocks start and end sooner, 16 rows at a time, each reading the cache again.
//   16 rows, few / tiles: one of 2000, 8000, 32000, 131072: 17 / 26, 22 / 30, 31 / 41, 90 / 83; 64 of 500: 36 / 54; 64 of
//   2000: 87 / 110; 16 of 3000: 48 / 48; 16 of 8192: 85 / 84; 32 heads of 64, 16 of 2000: 56 / 87 (32 rows: 79 / 91); 4 heads
//   of 256, 16 of 4000: 61 / 56.  Where it loses most, few / tiled: 16 of 500: 30 / 22; 16 of 1000: 34 / 30.
//   More rows, few / tiled, by the bytes of K that are read: 4 MB (one of 2000, 32 rows) 18 / 24; 8 MB (one of 2000, 64 rows)
//   20 / 24, (4 of 1000, 32 rows) 26 / 28; 16 MB (one of 8000, 32 rows) 24 / 26, (one of 4000, 64 rows) 22 / 25, (one of 2000,
//   128 rows) 28 / 26, (4 of 1000, 64 rows) 30 / 28, (16 of 500, 32 rows) 30 / 22.
// TILED, the kernel of prompts: 256 rows (head_dim 256: 128) that share the converted codes.
// TILES, the tree kernel: tiles of 64 or 128 rows in equal shares, which wins where they fill the card.  Tiles / tiled, by the
//   bytes of K, up to 64 rows: 17 MB (16 of 1000) 34 / 30, (one of 16000) 36 / 32; 33 MB (64 of 500) 67 / 71, (one of 32000)
//   44 / 44, (4 of 8192) 40 / 48; 50 MB (16 of 3000) 54 / 56; 134 MB (16 of 8192) 93 / 127, (one of 131072) 91 / 114.  Up to
//   128: 33 MB (64 of 500) 83 / 73, (4 of 8192) 48 / 46; 50 MB (16 of 3000) 68 / 58; 74 MB (32 heads of 64, 16 of 2000)
//   122 / 132; 135 MB (64 of 2000) 147 / 149, (16 of 8192) 123 / 128, (one of 131072) 120 / 115.
// The bounds decide, which the workspace's size follows from; a window, which that size is not asked with, has no say.
TreeKernel tree_kernel(int group, int kv_heads, int dim, int seqs, long long max_tokens, long long max_kv) {
    const long long rows = max_tokens * group;
    const double bytes = (double)seqs * kv_heads * (max_kv + max_tokens) * dim;
    if (rows <= (dim == 64 ? 32 : 16) || bytes * ((rows + kFewRows - 1) / kFewRows) <= 10e6) return TreeKernel::FEW;
    if (rows <= 64) return bytes < 25e6 ? TreeKernel::TILED : TreeKernel::TILES;
    return rows > 128 || dim == 256 || bytes < 60e6 ? TreeKernel::TILED : TreeKernel::TILES;
}

}  // namespace mmq

extern "C" {

mmq_status mmq_qk_norm_rope(const mmq_heads* q, int q_heads, const float* q_weight, const mmq_heads* q_out,
                            const mmq_heads* k, int k_heads, const float* k_weight, const mmq_heads* k_out,
                            int64_t tokens, int head_dim, const int32_t* positions, const mmq_rotary* rotary,
                            float eps, mmq_stream_t stream) {
    if (tokens < 0 || (!q && !k) || (!q != !q_out) || (!k != !k_out)) return MMQ_ERR_INVALID_ARG;
    if ((q && q_heads <= 0) || (k && k_heads <= 0)) return MMQ_ERR_INVALID_ARG;
    if (!head_dim_ok(head_dim) || tokens > kMaxDim) return MMQ_ERR_SHAPE;
    MMQ_TRY(check_rotary(rotary, head_dim));
    if (tokens == 0) return MMQ_OK;
    if (rotary && !positions) return MMQ_ERR_INVALID_ARG;
    for (const mmq_heads* r : {q, q_out, k, k_out})
        if (r) MMQ_TRY(check_rows(r));
    if (q && k && (q->dtype != k->dtype || q_out->dtype != k_out->dtype)) return MMQ_ERR_UNSUPPORTED;
    if (!aligned16(positions)) return MMQ_ERR_ALIGN;
    MMQ_TRY(check_weight(q_weight));
    MMQ_TRY(check_weight(k_weight));
    NormRopeArgs a{};
    a.q = rows_of(q);
    a.q_out = rows_of(q_out);
    a.k = rows_of(k);
    a.k_out = rows_of(k_out);
    a.q_weight = q ? q_weight : nullptr;
    a.k_weight = k ? k_weight : nullptr;
    a.q_heads = q ? q_heads : 0;
    a.k_heads = k ? k_heads : 0;
    a.tokens = (int)tokens;
    a.positions = positions;
    a.rot = rotary_of(rotary);
    a.eps = eps;
    return done(run_norm_rope(head_dim, (q ? q : k)->dtype, (q ? q_out : k_out)->dtype, a, stream_of(stream)),
                "mmq_qk_norm_rope");
}

mmq_status mmq_kv_append(const mmq_kv_cache* cache, const mmq_kv_seqs* seqs, int64_t tokens, const mmq_heads* k,
                         const mmq_heads* v, const float* k_weight, const mmq_heads* q, int q_heads,
                         const float* q_weight, const mmq_heads* q_out, const mmq_rotary* rotary, float eps,
                         mmq_stream_t stream) {
    return append(cache, seqs, nullptr, tokens, k, v, k_weight, q, q_heads, q_weight, q_out, rotary, eps,
                  stream_of(stream), "mmq_kv_append");
}

mmq_status mmq_kv_append_tree(const mmq_kv_cache* cache, const mmq_kv_seqs* seqs, const mmq_draft_tree* tree,
                              int64_t tokens, const mmq_heads* k, const mmq_heads* v, const float* k_weight,
                              const mmq_heads* q, int q_heads, const float* q_weight, const mmq_heads* q_out,
                              const mmq_rotary* rotary, float eps, mmq_stream_t stream) {
    if (!tree) return MMQ_ERR_INVALID_ARG;
    return append(cache, seqs, tree, tokens, k, v, k_weight, q, q_heads, q_weight, q_out, rotary, eps, stream_of(stream),
                  "mmq_kv_append_tree");
}

mmq_status mmq_kv_read(const mmq_kv_cache* cache, const mmq_kv_seqs* seqs, int64_t tokens, const mmq_heads* k_out,
                       const mmq_heads* v_out, mmq_stream_t stream) {
    MMQ_TRY(check_cache(cache));
    bool work;
    MMQ_TRY(check_seqs(seqs, tokens, &work));
    if (!k_out && !v_out) return MMQ_ERR_INVALID_ARG;
    if (!work) return MMQ_OK;
    if (k_out) MMQ_TRY(check_rows(k_out));
    if (v_out) MMQ_TRY(check_rows(v_out));
    if (k_out && v_out && k_out->dtype != v_out->dtype) return MMQ_ERR_UNSUPPORTED;
    ReadArgs a{};
    a.c = cache_of(cache);
    a.sq = seqs_of(seqs, tokens);
    a.k_out = rows_of(k_out);
    a.v_out = rows_of(v_out);
    return done(run_kv_read(cache->head_dim, (k_out ? k_out : v_out)->dtype, a, stream_of(stream)), "mmq_kv_read");
}

size_t mmq_attention_workspace_bytes(int64_t tokens, int n_heads, int kv_heads, int head_dim, int seqs,
                                     int64_t max_tokens, int64_t max_kv_len) {
    if (tokens <= 0 || n_heads <= 0 || kv_heads <= 0 || n_heads % kv_heads || !head_dim_ok(head_dim) || seqs <= 0 ||
        max_tokens <= 0 || max_kv_len < 0 || tokens > kMaxDim || tokens * n_heads > kMaxDim)
        return 0;
    if (max_tokens > tokens) max_tokens = tokens;
    return attention_plan(tokens, n_heads, kv_heads, head_dim, seqs, max_tokens, max_kv_len, 0).total;
}

mmq_status mmq_attention(const mmq_heads* q, int n_heads, const mmq_kv_cache* cache, const mmq_kv_seqs* seqs,
                         int64_t tokens, int64_t max_tokens, int64_t max_kv_len, float scale, int causal,
                         int64_t window, const mmq_heads* out, float* lse, void* workspace, size_t workspace_bytes,
                         mmq_stream_t stream) {
    MMQ_TRY(check_cache(cache));
    bool work;
    MMQ_TRY(check_seqs(seqs, tokens, &work));
    if (n_heads <= 0 || max_tokens < 0 || max_kv_len < 0 || window < 0 || (window > 0 && !causal) || !std::isfinite(scale))
        return MMQ_ERR_INVALID_ARG;
    if (n_heads % cache->kv_heads || tokens * n_heads > kMaxDim || max_kv_len > kMaxDim - 4096) return MMQ_ERR_SHAPE;
    if (!work) return MMQ_OK;
    if (max_tokens == 0) return MMQ_ERR_INVALID_ARG;
    MMQ_TRY(check_rows(q));
    MMQ_TRY(check_rows(out));
    if (q->dtype == MMQ_F32) return MMQ_ERR_UNSUPPORTED;
    if (!aligned16(lse)) return MMQ_ERR_ALIGN;
    if (max_tokens > tokens) max_tokens = tokens;
    const AttnPlan p = attention_plan(tokens, n_heads, cache->kv_heads, cache->head_dim, seqs->seqs, max_tokens,
                                      max_kv_len, window);
    const size_t need = mmq_attention_workspace_bytes(tokens, n_heads, cache->kv_heads, cache->head_dim, seqs->seqs,
                                                      max_tokens, max_kv_len);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MMQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MMQ_ERR_ALIGN;
    const AttnArgs a = attention_args(q, n_heads, cache, seqs, tokens, max_tokens, max_kv_len, scale, causal, p, out, lse, workspace);
    cudaStream_t s = stream_of(stream);
    cudaError_t e = p.few ? run_attention_few(cache->head_dim, q->dtype, out->dtype, a, p, s)
                          : run_attention_tiled(cache->head_dim, q->dtype, out->dtype, a, p, s);
    if (e == cudaSuccess && p.splits > 1) e = run_attention_join(cache->head_dim, out->dtype, a, p, s);
    return done(e, "mmq_attention");
}

mmq_status mmq_draft_masks(const int32_t* parents, const int32_t* cu_tokens, int32_t seqs, int64_t tokens,
                           int64_t max_tokens, int32_t* depths, uint32_t* masks, int32_t mask_words,
                           mmq_stream_t stream) {
    if (seqs < 0 || tokens < 0 || max_tokens < 0 || mask_words < 0) return MMQ_ERR_INVALID_ARG;
    if (tokens > kMaxDim || max_tokens > MMQ_MAX_DRAFT) return MMQ_ERR_SHAPE;
    if (!cu_tokens && tokens != seqs) return MMQ_ERR_INVALID_ARG;
    if (tokens == 0) return MMQ_OK;
    if (seqs == 0 || max_tokens == 0 || !parents || !depths || !masks) return MMQ_ERR_INVALID_ARG;
    if (mask_words < (max_tokens + 31) / 32 || mask_words * tokens > kMaxDim) return MMQ_ERR_SHAPE;
    if (!aligned16(parents) || !aligned16(cu_tokens) || !aligned16(depths) || !aligned16(masks)) return MMQ_ERR_ALIGN;
    const DraftArgs a{parents, cu_tokens, seqs, (int)tokens, (int)max_tokens, depths, masks, mask_words};
    return done(run_draft_masks(a, stream_of(stream)), "mmq_draft_masks");
}

mmq_status mmq_kv_keep(const mmq_kv_cache* cache, const mmq_kv_seqs* seqs, int64_t tokens, const int32_t* kept,
                       int64_t kept_stride, const int32_t* counts, mmq_stream_t stream) {
    MMQ_TRY(check_cache(cache));
    bool work;
    MMQ_TRY(check_seqs(seqs, tokens, &work));
    if (kept_stride < 0) return MMQ_ERR_INVALID_ARG;
    if (kept_stride > MMQ_MAX_DRAFT) return MMQ_ERR_SHAPE;
    if (!work) return MMQ_OK;
    if ((!kept && kept_stride > 0) || !counts) return MMQ_ERR_INVALID_ARG;
    if (!aligned16(kept) || !aligned16(counts)) return MMQ_ERR_ALIGN;
    const KeepArgs a{cache_of(cache), seqs_of(seqs, tokens), kept, counts, kept_stride};
    return done(run_kv_keep(cache->head_dim, a, stream_of(stream)), "mmq_kv_keep");
}

size_t mmq_attention_tree_workspace_bytes(int64_t tokens, int n_heads, int kv_heads, int head_dim, int seqs,
                                          int64_t max_tokens, int64_t max_kv_len) {
    if (tokens <= 0 || n_heads <= 0 || kv_heads <= 0 || n_heads % kv_heads || !head_dim_ok(head_dim) || seqs <= 0 ||
        max_tokens <= 0 || max_kv_len < 0 || max_kv_len > kMaxDim - 4096 || tokens > kMaxDim || tokens * n_heads > kMaxDim)
        return 0;
    if (max_tokens > tokens) max_tokens = tokens;
    if (max_tokens > MMQ_MAX_DRAFT) return 0;
    const TreeKernel kernel = tree_kernel(n_heads / kv_heads, kv_heads, head_dim, seqs, max_tokens, max_kv_len);
    if (kernel != TreeKernel::TILES)
        return attention_plan_of(kernel == TreeKernel::FEW, tokens, n_heads, kv_heads, head_dim, seqs, max_tokens, max_kv_len, 0)
            .total;
    const TreePlan p = tree_plan(n_heads, kv_heads, head_dim, seqs, max_tokens, max_kv_len);
    return p.fits ? p.total : 0;
}

mmq_status mmq_attention_tree(const mmq_heads* q, int n_heads, const mmq_kv_cache* cache, const mmq_kv_seqs* seqs,
                              const mmq_draft_tree* tree, int64_t tokens, int64_t max_tokens, int64_t max_kv_len,
                              float scale, int64_t window, const mmq_heads* out, float* lse, void* workspace,
                              size_t workspace_bytes, mmq_stream_t stream) {
    MMQ_TRY(check_cache(cache));
    bool work;
    MMQ_TRY(check_seqs(seqs, tokens, &work));
    if (!tree || n_heads <= 0 || max_tokens < 0 || max_kv_len < 0 || window < 0 || !std::isfinite(scale))
        return MMQ_ERR_INVALID_ARG;
    if (n_heads % cache->kv_heads || tokens * n_heads > kMaxDim || max_kv_len > kMaxDim - 4096) return MMQ_ERR_SHAPE;
    if (!work) return MMQ_OK;
    if (max_tokens == 0) return MMQ_ERR_INVALID_ARG;
    if (max_tokens > tokens) max_tokens = tokens;
    if (max_tokens > MMQ_MAX_DRAFT) return MMQ_ERR_SHAPE;
    MMQ_TRY(check_rows(q));
    MMQ_TRY(check_rows(out));
    if (q->dtype == MMQ_F32) return MMQ_ERR_UNSUPPORTED;
    if (!aligned16(lse)) return MMQ_ERR_ALIGN;
    const bool windowed = window > 0 && window < max_kv_len;
    if (windowed && window < max_tokens) return MMQ_ERR_UNSUPPORTED;
    if (!tree->masks || (windowed && !tree->depths)) return MMQ_ERR_INVALID_ARG;
    if (tree->mask_words < (max_tokens + 31) / 32 || tree->mask_words * tokens > kMaxDim) return MMQ_ERR_SHAPE;
    if (!aligned16(tree->masks) || !aligned16(tree->depths)) return MMQ_ERR_ALIGN;
    const int group = n_heads / cache->kv_heads;
    const TreeKernel kernel = tree_kernel(group, cache->kv_heads, cache->head_dim, seqs->seqs, max_tokens, max_kv_len);
    const TreePlan p = tree_plan(n_heads, cache->kv_heads, cache->head_dim, seqs->seqs, max_tokens, max_kv_len);
    if (kernel == TreeKernel::TILES && !p.fits) return MMQ_ERR_SHAPE;
    const size_t need = mmq_attention_tree_workspace_bytes(tokens, n_heads, cache->kv_heads, cache->head_dim, seqs->seqs,
                                                           max_tokens, max_kv_len);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MMQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MMQ_ERR_ALIGN;
    cudaStream_t s = stream_of(stream);
    if (kernel != TreeKernel::TILES) {
        const AttnPlan fp = attention_plan_of(kernel == TreeKernel::FEW, tokens, n_heads, cache->kv_heads, cache->head_dim,
                                              seqs->seqs, max_tokens, max_kv_len, windowed ? window : 0);
        AttnArgs a = attention_args(q, n_heads, cache, seqs, tokens, max_tokens, max_kv_len, scale, 1, fp, out, lse, workspace);
        a.depths = tree->depths;
        a.masks = tree->masks;
        a.words = tree->mask_words;
        cudaError_t e = fp.few ? run_attention_few(cache->head_dim, q->dtype, out->dtype, a, fp, s)
                               : run_attention_tiled(cache->head_dim, q->dtype, out->dtype, a, fp, s);
        if (e == cudaSuccess && fp.splits > 1) e = run_attention_join(cache->head_dim, out->dtype, a, fp, s);
        return done(e, "mmq_attention_tree");
    }
    TreeArgs a{};
    a.q = rows_of(q);
    a.out = rows_of(out);
    a.c = cache_of(cache);
    a.sq = seqs_of(seqs, tokens);
    a.depths = tree->depths;
    a.masks = tree->masks;
    a.words = tree->mask_words;
    a.heads = n_heads;
    a.group = group;
    a.max_tokens = (int)max_tokens;
    a.max_kv = (int)max_kv_len;
    a.scale = scale;
    a.window = windowed ? (int)window : 0;
    a.lse = lse;
    return done(run_attention_tree(cache->head_dim, q->dtype, out->dtype, a, p, workspace, s),
                "mmq_attention_tree");
}

}  // extern "C"
