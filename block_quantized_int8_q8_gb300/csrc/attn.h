// attn.h -- host-side interface between the attention boundary (attn_api.cu) and its kernels: norm and
// rotation, the quantizing append, the cache read (kv_cache.cu), attention of few rows (attn_few.cu)
// and of prompts (attn_tiled.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include "../../include/mmq.h"

namespace mmq {

// Rows of heads with byte-sized strides left in elements.
struct HeadRows {
    void* data;
    long long ts, hs;          // token and head stride, elements
};

struct RotaryArgs {
    const float* cos;          // null: no rotation
    const float* sin;
    long long positions;
    int half;                  // rot_dim / 2
    int interleaved;
};

struct CacheArgs {
    int8_t* k;
    int8_t* v;
    float* ks;
    float* vs;
    long long pages;
    int heads, page, block;
};

struct SeqArgs {
    const int32_t* table;
    long long stride;          // entries of a table row
    const int32_t* lens;
    const int32_t* cu;         // null: token t is sequence t
    int seqs;
    int tokens;
};

struct NormRopeArgs {
    HeadRows q, q_out, k, k_out;
    const float* q_weight;
    const float* k_weight;
    int q_heads, k_heads, tokens;
    const int32_t* positions;
    RotaryArgs rot;
    float eps;
};
cudaError_t run_norm_rope(int dim, mmq_dtype it, mmq_dtype ot, const NormRopeArgs& a,
                          cudaStream_t s);

struct AppendArgs {
    CacheArgs c;
    SeqArgs sq;
    HeadRows k, v, q, q_out;
    const float* k_weight;
    const float* q_weight;
    int q_heads;               // 0: no queries
    RotaryArgs rot;
    float eps;
    const int32_t* depths;     // null: a token turns at its place, else at this many past the cached text
};
cudaError_t run_kv_append(int dim, mmq_dtype t, mmq_dtype qot, const AppendArgs& a, cudaStream_t s);

struct ReadArgs {
    CacheArgs c;
    SeqArgs sq;
    HeadRows k_out, v_out;     // data null: not wanted
};
cudaError_t run_kv_read(int dim, mmq_dtype t, const ReadArgs& a, cudaStream_t s);

struct AttnArgs {
    HeadRows q, out;
    CacheArgs c;
    SeqArgs sq;
    int heads, group;          // query heads; query heads per key/value head
    int max_tokens, max_kv;
    float scale;
    int causal, window;        // window 0: none
    float* lse;
    // split along the cache, or a part longer than kChain: sums of rows [split][row] (row = token * heads + head)
    float* part_o;             // [splits][rows][dim], not divided by the denominator
    float2* part_ml;           // [splits][rows]: running maximum (log2) and denominator
    // a tree of drafted tokens: null masks where there is none; words of a row of masks
    const int32_t* depths;
    const uint32_t* masks;
    int words;
};
// Most tokens that the tiled kernel sums in one go.
constexpr int kChain = 32768;
// Thread blocks of the few-row kernel that fit on an SM (its launch bound), for head_dim and 8 or 16 rows.
constexpr int few_blocks(int dim, int nt) { return dim == 256 ? 2 : (nt == 2 ? 3 : 4); }
// How a problem is split along the cache: chunk tokens per part, and the parts of the longest sequence.
struct AttnPlan {
    bool few;                  // the few-row kernel, else the tiled one
    int chunk, splits;
    int window;                // 0 where the asked one hides nothing: what the kernels are given
    size_t part_o, part_ml, total;     // workspace offsets and size
};
// Most rows (new tokens x query heads) of a key/value head that the few-row kernel takes at once.
constexpr int kFewRows = 16;
AttnPlan attention_plan(long long tokens, int heads, int kv_heads, int dim, int seqs, long long max_tokens,
                        long long max_kv, long long window);
// The same for the kernel that is asked for.
AttnPlan attention_plan_of(bool few, long long tokens, int heads, int kv_heads, int dim, int seqs, long long max_tokens,
                           long long max_kv, long long window);
cudaError_t run_attention_few(int dim, mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p,
                              cudaStream_t s);
cudaError_t run_attention_tiled(int dim, mmq_dtype qt, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p,
                                cudaStream_t s);
// Joins the parts of rows whose cache range was split (attn_few.cu).
cudaError_t run_attention_join(int dim, mmq_dtype ot, const AttnArgs& a, const AttnPlan& p, cudaStream_t s);

// Trees of drafted tokens (draft.cu).
struct DraftArgs {
    const int32_t* parents;
    const int32_t* cu;         // null: token t is sequence t
    int seqs, tokens, max_tokens;
    int32_t* depths;
    uint32_t* masks;
    int words;                 // of a row of masks
};
cudaError_t run_draft_masks(const DraftArgs& a, cudaStream_t s);

struct KeepArgs {
    CacheArgs c;
    SeqArgs sq;
    const int32_t* kept;       // [seqs][stride] rows, of which counts[s] count
    const int32_t* counts;
    long long stride;
};
cudaError_t run_kv_keep(int dim, const KeepArgs& a, cudaStream_t s);

// Which kernel a tree's rows take (attn_api.cu): the few-row kernel, attn_tree.cu's, the kernel of prompts.
enum class TreeKernel { FEW, TILES, TILED };
TreeKernel tree_kernel(int group, int kv_heads, int dim, int seqs, long long max_tokens, long long max_kv);

// Attention of 17 to 128 rows of a tree (head_dim 256: 64) over long texts (attn_tree.cu).
struct TreeArgs {
    HeadRows q, out;
    CacheArgs c;
    SeqArgs sq;
    const int32_t* depths;
    const uint32_t* masks;
    int words;
    int heads, group;
    int max_tokens, max_kv;
    float scale;
    int window;                // 0: none
    float* lse;
};
// How a problem is shared out: rows that a tile has room for, workspace offsets and size.
struct TreePlan {
    int rows;
    bool many_parts;           // a unit is cut into many
    bool fits;                 // positions in the line of tiles are 32-bit numbers
    size_t joins, part_ml, part_o, total;
};
TreePlan tree_plan(int heads, int kv_heads, int dim, int seqs, long long max_tokens, long long max_kv);
cudaError_t run_attention_tree(int dim, mmq_dtype qt, mmq_dtype ot, const TreeArgs& a, const TreePlan& p, void* workspace,
                               cudaStream_t s);

cudaError_t read_clear_errors_draft(unsigned* bits, cudaStream_t s);
cudaError_t read_clear_errors_attn_tree(unsigned* bits, cudaStream_t s);
cudaError_t read_clear_errors_kv_cache(unsigned* bits, cudaStream_t s);
cudaError_t read_clear_errors_attn_few(unsigned* bits, cudaStream_t s);
cudaError_t read_clear_errors_attn_tiled(unsigned* bits, cudaStream_t s);

}  // namespace mmq
