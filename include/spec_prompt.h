/*
 * spec_prompt.h -- C ABI of libspecverify: attention of whole prompts over
 * themselves, next to the cache of spec_cache.h (which a prompt's keys and values
 * enter by spec_cache_append, and over which steps of up to 32 rows attend).
 *
 * Conventions are those of spec_verify.h: device pointers owned by the
 * caller, asynchronous on `stream`, no allocation, argument errors returned
 * before any launch, problems in device data OR-ed into *status.  Arrays are
 * aligned to their type, the workspace to 16 bytes; anything else is refused.
 */
#ifndef SPEC_PROMPT_H
#define SPEC_PROMPT_H

#include "spec_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_PROMPT_MOST_KEYS (1 << 24)      /* keys of a call, of all requests */

/* Packed prompts: request b's rows are cu_rows[b] .. cu_rows[b+1]-1 of q and out, its
 * keys cu_keys[b] .. cu_keys[b+1]-1 of k and v.  Its rows are the last of its keys: with
 * n rows and m >= n keys (a piece of a prompt over what came before) row i is key m - n + i. */
typedef struct {
    const void *q;             /* [R_cap] rows of [Hq] heads of D channels, unit channel stride */
    const void *k, *v;         /* [K_cap] rows of [H] heads of D channels, unit channel stride  */
    int32_t dtype;             /* spec_dtype of q, k, v and out                               */
    int32_t D;                 /* channels of a head: 64, 128 or 256                          */
    int32_t Hq, H;             /* query heads, a multiple of the kv heads H >= 1: head h reads
                                  kv head h/(Hq/H)                                            */
    int64_t q_row, q_head;     /* strides in elements                                         */
    int64_t k_row, k_head;
    int64_t v_row, v_head;
    int32_t B;                 /* requests, >= 1                                              */
    int32_t R_cap, K_cap;      /* host-known bounds on cu_rows[B], cu_keys[B], >= 1; K_cap at
                                  most SPEC_PROMPT_MOST_KEYS                                   */
    const int32_t *cu_rows;    /* [B+1]                                                       */
    const int32_t *cu_keys;    /* [B+1] or NULL: cu_rows                                      */
    float scale;               /* of q . k; finite, and so times log2(e)                      */
    float cap;                 /* > 0: s = cap * tanh(s / cap) (above 2^120: as 2^120); 0: off */
    const float *slopes;       /* [Hq] or NULL: s -= slope * (row's key - key)                */
    int32_t window;            /* > 0: only keys less than `window` before the row's own ...   */
    int32_t prefix;            /* ... or among the first `prefix`                             */
    uint32_t *status;          /* [1] or NULL                                                 */
} spec_prompt;

/* Workspace of spec_prompt_attend, 16-byte aligned, zero-filled once before its first use;
 * any number of stream-ordered calls, of any shapes that it is large enough for, can then
 * share it (after SPEC_STATUS_TIMEOUT it has to be zeroed again).  0 for invalid sizes. */
SPEC_API size_t spec_prompt_workspace_bytes(int32_t Hq, int32_t H, int32_t D, int32_t dtype);

/*
 * out[r][h] = sum_j softmax_j(s_rj) v_j and lse[r][h] = log sum_j exp(s_rj)
 * (natural, fp32) over the keys j that row r sees: those up to its own, with
 * window > 0 only the nearest `window` of them and the first `prefix`.  A row that sees
 * no key (m < n) gets out = 0 and lse = -inf, as do all rows of a request with malformed
 * cu_keys (SPEC_STATUS_BAD_LENGTH).  out [R_cap, Hq, D] and lse [R_cap, Hq] or NULL, both
 * contiguous; rows >= cu_rows[B], and those of a request with malformed cu_rows
 * (SPEC_STATUS_BAD_ROWS), are not written; where offsets go back, so that rows lie in two requests, those may hold either's
 * results or be left, and rows of the requests after them may be left too.  Keys and values that no row of their request
 * sees may hold anything; those that one of its rows sees have to be finite, as have
 * the queries (a row of another request never notices).  The scores, times log2(e), have to stay within
 * fp32, and values below 2^95 (2^24 of them, with weights of up to 2^8, are added up in fp32).  Results do not depend on the order in which blocks run; into how many parts a bf16 row's keys are split goes by B, R_cap, K_cap,
 * the heads, D, the options and the GPU, so that its last bits can be others in a padded or a larger batch.
 * out and lse must not overlap the inputs.
 * bf16: products of bf16 in fp32, weights rounded to bf16 (8 bits) before they meet the values,
 * their sums, and so lse, in fp32, as are the sums of values, which lose up to 2^-12 of themselves to truncation.  They run on the tensor cores where q, k and v start on 16 bytes, their
 * strides are positive multiples of 16 bytes, out starts on 16 bytes and Hq / H is at most 128; on the CUDA
 * cores, many times slower, elsewhere, then with weights in fp32.  f32: fp32 throughout.  On the CUDA cores the sums of
 * weights and of values lose at most 2^-17 of their terms' magnitudes to roundings, over any number of keys.
 */
SPEC_API int spec_prompt_attend(const spec_prompt *prompt, void *out, float *lse, void *workspace,
                                size_t workspace_bytes, spec_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_PROMPT_H */
