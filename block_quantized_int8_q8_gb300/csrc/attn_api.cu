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
    AttnPlan p{};
    constexpr long long SMS = 152;
    const long long rows = max_tokens * (heads / kv_heads);
    p.few = rows <= 16;
    const long long pairs = (long long)seqs * kv_heads, granule = p.few ? 64 : 128;
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
    MMQ_TRY(check_cache(cache));
    bool work;
    MMQ_TRY(check_seqs(seqs, tokens, &work));
    MMQ_TRY(check_rotary(rotary, cache->head_dim));
    if (!q != !q_out || (q && q_heads <= 0)) return MMQ_ERR_INVALID_ARG;
    if (!work) return MMQ_OK;
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
    return done(run_kv_append(cache->head_dim, k->dtype, q ? q_out->dtype : k->dtype, a, stream_of(stream)),
                "mmq_kv_append");
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
    cudaStream_t s = stream_of(stream);
    cudaError_t e = p.few ? run_attention_few(cache->head_dim, q->dtype, out->dtype, a, p, s)
                          : run_attention_tiled(cache->head_dim, q->dtype, out->dtype, a, p, s);
    if (e == cudaSuccess && p.splits > 1) e = run_attention_join(cache->head_dim, out->dtype, a, p, s);
    return done(e, "mmq_attention");
}

}  // extern "C"
