// internal.h -- declarations shared by the translation units of libspecverify.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace specv {

enum Mode : int { MODE_GREEDY = 0, MODE_RELAXED = 1, MODE_SAMPLE = 2, MODE_CONF = 3 };

// Workspace of the row kernel, per packed row r and chunk c (a row is split
// into nchunk = ceil(V * elt / kChunkBytes) chunks, one work item each):
//   info[r]     (64 bytes) owner request and parameters of the row
//   part[r][c]  (32 bytes) chunk reduction and sampler summary
//   cand[r][c]  (kWsCandCap (value, index) pairs) candidate lists, or for
//               bf16 top-p alone the listed elements and value counts
//                                                             (sampler only)
constexpr int kWsCandCap = 512;

// Everything one verify launch needs (passed by value to the row kernel).
struct VerifyParams {
    const void *logits;
    int64_t ld;
    int32_t V, B, k_max, R_cap;
    const int32_t *cu_rows;      // [B+1]        (not used by MODE_CONF)
    const int32_t *draft_ids;    // [R_cap]
    // stochastic verification
    const float *temperature;
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
    const uint64_t *seed;
    const uint32_t *request_id;
    uint32_t step;
    // relaxed top-K
    const int32_t *relaxed_k;
    // greedy with a confidence margin (margin == nullptr: strict greedy)
    const float *margin;
    const int32_t *generated;
    const int32_t *protected_ids;
    int32_t n_protected, from_position, after_tokens;
    // greedy over an active vocabulary: full token id of each column (or nullptr)
    const int32_t *vocab_ids;
    // draft confidence (MODE_CONF: rows are draft positions)
    const int32_t *selected;
    float *conf;
    int32_t *draft_token;
    // request outputs
    int32_t *accepted_len;
    int32_t *out_tokens;
    int32_t *next_token;
    // optional row outputs
    float *row_max;
    float *row_lse;
    int32_t *row_argmax;
    int32_t *row_token;
    uint32_t *status;
    // optional fused prefix statistics
    int64_t *acc;
    int64_t *ver;
    int64_t *hist;
    // workspace
    int32_t *ws_tok;             // [R_cap] per-row target token
    int32_t *ws_flag;            // [R_cap] per-row relaxed acceptance
    uint32_t *ws_ticket;         // [B] arrivals per request (zero between calls)
    void *ws_info;               // [R_cap] row records (64 bytes each)
    void *ws_part;               // [R_cap * nchunk] chunk partials (32 bytes each)
    void *ws_cand;               // [R_cap * nchunk * kWsCandCap] (value, index) pairs
    int32_t nchunk;              // chunks per row
    int32_t n_rows;              // rows of the work (R_cap; draft rows for the confidence)
};

struct AllocParams {
    const float *conf;
    const int32_t *draft_token;
    int32_t B, k;
    float threshold;
    int32_t max_rows;
    int32_t *k_alloc;
    int32_t *cu_rows;
    int32_t *row_owner;
    int32_t *row_pos;
    int32_t *packed_draft;
    int32_t *total_rows;
    uint32_t *status;
};

// ---- the 4-bit paged cache (include/spec_cache.h) ----

// The cache as a batch of requests sees it (passed by value to the kernels).
struct CacheView {
    uint8_t *pages;
    int64_t n_pages;
    int32_t page_tokens, H, D;
    const float *k_scale, *v_scale;
    int32_t B, max_pages;
    const int32_t *page_table;
};

// Rows entering (append) or leaving (read) the cache.
struct CacheRows {
    void *k, *v;
    int64_t k_row, k_head, v_row, v_head;
    int32_t R_cap, max_rows;
    const int32_t *cu_rows, *start;
    float *score;
    int32_t *slot_pos;
    const int32_t *pos0;
    uint32_t *status;
    bool k_aligned, v_aligned;   // every head's first channel lies on a 16-byte boundary
};

struct AttnParams {
    const void *q;
    int64_t q_row, q_head;
    int32_t Hq, R_cap, k_max;
    const int32_t *cu_rows, *len;
    int32_t max_len;
    float scale, cap;
    float scale_log2;            // |scale| log2 e, rounded once
    const float *slopes;
    int32_t window, prefix;
    const int32_t *slot_pos;
    uint32_t *status;
    void *out;
    float *lse;                  // attend: written; weights: read
    float *score;                // weights only
    const int32_t *parent;       // the rows as a tree (or null: a chain)
    void *ws;
    bool q_aligned;              // every query starts on a 16-byte boundary
};

// Whole prompts over themselves (include/spec_prompt.h).
struct PromptParams {
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    int32_t Hq, H, D, B, R_cap, K_cap;
    const int32_t *cu_rows, *cu_keys;    // cu_keys null: cu_rows
    float scale, cap;
    const float *slopes;
    int32_t window, prefix;
    uint32_t *status;
    void *out;
    float *lse;
    void *ws;
    bool q_aligned, k_aligned, v_aligned;    // every head starts on a 16-byte boundary
};

// Trees of drafts and the adjustment of logits (include/spec_tree.h).
struct TreeParams {
    int32_t B, k_max, R_cap;
    const int32_t *cu_rows, *row_token, *node_token, *parent;
    int32_t *accepted_len, *out_tokens, *next_token, *path_rows;
    uint32_t *status;
};

struct LogitParams {
    const void *logits;
    int64_t ld;
    int32_t V, B, k_max, R_cap;
    const int32_t *cu_rows;
    const int32_t *history;
    int64_t history_ld;
    int32_t history_cap;
    const int32_t *n_tokens, *n_prompt;
    const float *repetition, *frequency, *presence;
    const int32_t *node_token, *parent;
    const int32_t *bias_cu, *bias_ids;
    const float *bias_values;
    int32_t n_bias;
    const uint32_t *allowed;
    int64_t allowed_ld;
    int32_t n_allowed;
    const int32_t *allowed_row;
    uint32_t *status;
    void *out;
    int64_t out_ld;
};

struct EvictParams {
    float *score;
    int32_t *slot_pos;
    const int32_t *len;
    int32_t budget, recent;
    const int32_t *dst_table;
    int32_t dst_pages;
    int32_t *kept, *new_len;
    uint32_t *status;
};

cudaError_t launch_cache_rows(const CacheView &c, const CacheRows &r, int dtype, bool append,
                              cudaStream_t stream);
cudaError_t launch_cache_attend(const CacheView &c, const AttnParams &p, int dtype,
                                cudaStream_t stream);
// the same with a cap, distance biases or a window, and for trees of rows (called by
// launch_cache_attend)
cudaError_t launch_cache_attend_options(const CacheView &c, const AttnParams &p, int dtype,
                                        cudaStream_t stream);
cudaError_t launch_cache_attend_tree(const CacheView &c, const AttnParams &p, int dtype,
                                     cudaStream_t stream);
cudaError_t launch_cache_attend_tree_options(const CacheView &c, const AttnParams &p, int dtype,
                                             cudaStream_t stream);
cudaError_t launch_cache_weights(const CacheView &c, const AttnParams &p, int dtype,
                                 cudaStream_t stream);
// workspace bytes of the attention (for queries of either type)
size_t cache_attend_workspace(int B, int k_max, int Hq, int H, int D, int max_len);
// attention of prompts, and its workspace
cudaError_t launch_prompt(const PromptParams &p, int dtype, cudaStream_t stream);
size_t prompt_workspace(int D, int dtype);
// on the CUDA cores, either type (called by launch_prompt)
cudaError_t launch_prompt_rows(const PromptParams &p, int dtype, cudaStream_t stream);
cudaError_t launch_tree_accept(const TreeParams &p, cudaStream_t stream);
cudaError_t launch_adjust_logits(const LogitParams &p, int dtype, cudaStream_t stream);
cudaError_t launch_cache_evict(const CacheView &c, const EvictParams &p, cudaStream_t stream);

// Host launchers (return cudaError_t of the launch).
cudaError_t launch_verify(int mode, int dtype, const VerifyParams &p, cudaStream_t stream);
// the row path of relaxed top-K (bf16, large batches; called by launch_verify)
cudaError_t launch_relaxed_rows(const VerifyParams &p, cudaStream_t stream);
cudaError_t launch_alloc(const AllocParams &p, cudaStream_t stream);
cudaError_t launch_restore_rows(const void *src, int64_t src_ld, int32_t R_cap,
                                const int32_t *cu_rows, int32_t B, int32_t k_max,
                                int64_t row_bytes, void *dst, int64_t dst_ld, uint32_t *status,
                                cudaStream_t stream);
cudaError_t launch_prefix_stats(const int32_t *accepted_len, const int32_t *cu_rows, int32_t B,
                                int32_t k_max, int64_t *acc, int64_t *ver, int64_t *hist,
                                uint32_t *status, cudaStream_t stream);

// Largest row (bytes) the verify path accepts.
size_t max_row_bytes();

// chunks per row for a vocabulary of V elements of `elt` bytes
int chunks_per_row(int32_t V, int elt);

// workspace bytes of the row kernel (sampling adds the candidate lists)
size_t row_workspace_bytes(int32_t R_cap, int32_t B, int32_t V, int elt, bool sampling);

}  // namespace specv
