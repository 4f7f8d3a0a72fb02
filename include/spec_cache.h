/*
 * spec_cache.h -- C ABI of libspecverify: the target model's key/value cache
 * in 4 bits, next to the verification of spec_verify.h: append a step's rows,
 * attend over the cache with the packed verify rows, accumulate attention
 * weights, evict the tokens that got the least.
 *
 * One speculative step of a request with k_b drafts appends k_b + 1 keys and
 * values (spec_cache_append), attends with its k_b + 1 rows
 * (spec_cache_attend), verifies, and keeps the accepted prefix by setting its
 * cache length to old length + a_b + 1: rejected slots are overwritten by the
 * next append.  The rows are packed by cu_rows exactly as in spec_verify.h.
 *
 * The cache.  A pool of n_pages pages of page_tokens tokens (a multiple of
 * 32); the pages of a request are named by its row of page_table.  A page is
 * [kv head][block of 32 tokens][36 * D bytes], and a block holds
 *     K codes   [D/32][32 tokens][16 B]  byte j of a chunk: channels 2j, 2j+1
 *     K scales  [32 tokens][D/16 B]      e4m3, one per 16 channels of a token
 *     V codes   [D][16 B]                byte j of a channel: tokens 2j, 2j+1
 *     V scales  [D/16][32 tokens]        e4m3, one per 16 channels of a token
 * (the first of two codes in the low nibble).  A code is e2m1 (magnitudes 0,
 * 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit); a value is code * scale * g, where
 * g is the kv head's k_scale / v_scale (1 when NULL).  Keys lie token by
 * token and values channel by channel because that is how the two matrix
 * products over the cache read them.
 *
 * Conventions are those of spec_verify.h: device pointers owned by the
 * caller, asynchronous on `stream`, no allocation, argument errors returned
 * before any launch, problems in device data OR-ed into *status.  Arrays are
 * aligned to their type, pages and workspace to 16 bytes; anything else is refused.
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_CACHE_BLOCK_TOKENS 32

/* further device status bits */
#define SPEC_STATUS_BAD_PAGE   0x400u  /* page id outside [0, n_pages): its tokens are hidden / skipped */
#define SPEC_STATUS_BAD_LENGTH 0x800u  /* length outside [0, max_pages * page_tokens] (attention: [0,
                                          max_len]): request skipped; its rows see nothing        */

/* The cache as a batch of B requests sees it. */
typedef struct {
    void *pages;               /* [n_pages][H][page_tokens/32][36 D] bytes, 16-byte aligned   */
    int64_t n_pages;
    int32_t page_tokens;       /* a multiple of 32, at most 65536                             */
    int32_t H;                 /* kv heads, >= 1                                              */
    int32_t D;                 /* channels of a head: 64, 128 or 256                          */
    const float *k_scale;      /* [H] or NULL: head scale of the keys, finite and > 0         */
    const float *v_scale;      /* [H] or NULL: head scale of the values                       */
    int32_t B;                 /* requests, >= 1                                              */
    int32_t max_pages;         /* row length of page_table                                    */
    const int32_t *page_table; /* [B, max_pages]; entries past a request's length are unread  */
} spec_cache;

/* Rows entering or leaving the cache. */
typedef struct {
    void *k, *v;               /* [R_cap] rows of [H] heads of D channels, unit channel stride */
    int32_t dtype;             /* spec_dtype                                                  */
    int64_t k_row, k_head;     /* strides of k in elements                                    */
    int64_t v_row, v_head;
    int32_t R_cap;             /* host-known bound on cu_rows[B]                              */
    int32_t max_rows;          /* host-known bound on one request's rows, >= 1                */
    const int32_t *cu_rows;    /* [B+1]                                                       */
    const int32_t *start;      /* [B] cache slot of each request's first row                  */
    float *score;              /* append: [n_pages, page_tokens] or NULL: 0 at the new slots  */
    int32_t *slot_pos;         /* append: [n_pages, page_tokens] or NULL: positions written   */
    const int32_t *pos0;       /* append: [B] or NULL (= start): position of the first row    */
    uint32_t *status;          /* [1] or NULL                                                 */
} spec_cache_rows;

/*
 * Quantise the rows and write them to slots start[b] .. start[b] + n_b - 1 of
 * their requests.  Per 16 channels, in fp32 with IEEE rounding:
 *   s = e4m3(min(max|x| / (6 g), 448)),  code = e2m1(x / (s g)),
 * both rounded to nearest even (codes saturate at 6; s = 0 gives code 0).
 * Other slots keep their bytes.  A request's pages must be its own: two
 * requests that append to one block race.  The values must be finite.
 * Malformed cu_rows (n_b < 0, n_b > max_rows, rows outside [0, R_cap]) skip
 * the request and set SPEC_STATUS_BAD_ROWS; a slot past the page table,
 * SPEC_STATUS_BAD_LENGTH; a page id out of range skips its rows.
 * One launch; the rows are read once.
 */
SPEC_API int spec_cache_append(const spec_cache *cache, const spec_cache_rows *rows,
                               spec_stream stream);

/*
 * The inverse: the values that slots start[b] .. start[b] + n_b - 1 stand for,
 * code * s (exact) * g, rounded once to `dtype`.  Rows of a bad page come out
 * as zeros; rows of a skipped request are not written.
 */
SPEC_API int spec_cache_read(const spec_cache *cache, const spec_cache_rows *rows,
                             spec_stream stream);

/* Attention of packed rows over the cache. */
typedef struct {
    const void *q;             /* [R_cap] rows of [Hq] heads of D channels, unit channel stride */
    int32_t dtype;             /* spec_dtype of q and out                                     */
    int64_t q_row, q_head;     /* strides in elements                                         */
    int32_t Hq;                /* query heads, a multiple of H: head h reads kv head h/(Hq/H) */
    int32_t R_cap;
    int32_t k_max;             /* at most k_max + 1 rows a request, 0..31                     */
    const int32_t *cu_rows;    /* [B+1]                                                       */
    const int32_t *len;        /* [B] tokens in the cache, this step's rows included          */
    int32_t max_len;           /* host-known bound on len (0: max_pages * page_tokens)        */
    float scale;               /* of q . k; finite, and so times log2(e)                      */
    float cap;                 /* > 0: s = cap * tanh(s / cap) (above 2^120: as 2^120); 0: off */
    const float *slopes;       /* [Hq] or NULL: s -= slope * (pos_row - pos_slot)             */
    int32_t window;            /* > 0: only slots with pos_row - pos_slot < window ...        */
    int32_t prefix;            /* ... or slot < prefix                                        */
    const int32_t *slot_pos;   /* [n_pages, page_tokens] or NULL: position of a slot, not
                                  decreasing over a request's slots, the last less than 2^31
                                  beyond the first; NULL: its index                           */
    uint32_t *status;          /* [1] or NULL                                                 */
} spec_attention;

/* Workspace of spec_cache_attend, 16-byte aligned, zero-filled once before its first use; any
 * number of stream-ordered calls, of any shapes that it is large enough for, can
 * then share it (after SPEC_STATUS_TIMEOUT it has to be zeroed again).  0 for
 * invalid sizes. */
SPEC_API size_t spec_cache_workspace_bytes(int32_t B, int32_t k_max, int32_t Hq, int32_t H,
                                           int32_t D, int32_t max_len);

/*
 * out[r][h] = sum_j softmax_j(s_rj) v_j and lse[r][h] = log sum_j exp(s_rj)
 * (natural, fp32) over the slots j that row r of request b sees:
 * j <= len_b - n_b + (r - cu_rows[b]), its own slot, so the rows of a step are
 * causal among themselves; with window > 0 also pos - pos_j < window or
 * j < prefix.  A row that sees no slot (a window that hides all, len_b < n_b,
 * a bad length) gets out = 0 and lse = -inf.  What slots hold that no row of the
 * request sees does not matter, NaN scales included (the scales of the others have
 * to be numbers).  Pages whose slots a window hides from all rows can be given back
 * and need no id: their entries are not looked at, and with slot_pos, where only
 * positions tell, bad ids that follow hidden slots (or begin the cache, with
 * position 0 hidden) count as such and are not reported.  out [R_cap, Hq, D], lse
 * [R_cap, Hq] or NULL, both contiguous; rows >= cu_rows[B], and those of a request
 * with malformed cu_rows (SPEC_STATUS_BAD_ROWS), are not written.
 * Results do not depend on the order in which blocks run.  A query row with a
 * NaN or infinite value gets unspecified results, as can the request's other rows
 * of the same kv head; every other row its own.  One launch.  bf16
 * outputs come from weights rounded to 11 bits, fp32 ones from 22 bits; sums of
 * weights, and so lse, are fp32, and so are the sums of values, of which bf16's lose
 * up to 2^-13 of themselves to truncation, over a cache of any length.
 */
SPEC_API int spec_cache_attend(const spec_cache *cache, const spec_attention *attn, void *out,
                               float *lse, void *workspace, size_t workspace_bytes,
                               spec_stream stream);

/*
 * The same where a request's rows are the nodes of a tree: parent [R_cap] as in spec_tree.h.
 * Row i of request b sees the slots before the step's, j < len_b - n_b, of the step's slots those of its
 * ancestors and its own, and no others.  Its position is that of the root's slot plus its depth (a
 * row that hangs on no other has depth 0), and so is its slot's, for slopes and window: with slot_pos, only
 * the root's entry is read of the step's slots.  With len_b < n_b its rows see nothing
 * (SPEC_STATUS_BAD_LENGTH).  Workspace as for spec_cache_attend; it may be shared.
 */
SPEC_API int spec_cache_attend_tree(const spec_cache *cache, const spec_attention *attn,
                                    const int32_t *parent, void *out, float *lse, void *workspace,
                                    size_t workspace_bytes, spec_stream stream);

/*
 * score[slot] += sum over the request's rows r and all query heads h of
 * exp(s_rj - lse[r][h]) for every slot j that some row sees (s, masks and lse
 * as in spec_cache_attend): the attention each cached token got this step.  Rows
 * with lse = -inf count 0: those that saw nothing, and those that the caller marks
 * so, as it should the rows of rejected drafts before weights that eviction goes by.  score [n_pages, page_tokens].  A request's sum runs in a
 * fixed order and is added to the slot's score once; requests that share a page (a
 * common prompt) all count, and which of them adds first is open: there, and there
 * alone, the last place can change from call to call.
 */
SPEC_API int spec_cache_weights(const spec_cache *cache, const spec_attention *attn,
                                const float *lse, float *score, spec_stream stream);

/* Eviction. */
typedef struct {
    float *score;              /* [n_pages, page_tokens] accumulated weights                  */
    int32_t *slot_pos;         /* [n_pages, page_tokens] or NULL                              */
    const int32_t *len;        /* [B]                                                         */
    int32_t budget;            /* tokens kept per request, >= 1                               */
    int32_t recent;            /* the newest slots, always kept, 0..budget                    */
    const int32_t *dst_table;  /* [B, dst_pages] pages that receive the kept tokens           */
    int32_t dst_pages;
    int32_t *kept;             /* [B, budget] kept slots, ascending, -1 padded                */
    int32_t *new_len;          /* [B] min(len, budget); can be len itself                     */
    uint32_t *status;          /* [1] or NULL                                                 */
} spec_eviction;

/*
 * Keep of each request the `recent` newest slots and, of the others, those
 * with the highest score (ties: the lowest slot; NaN below everything) up to
 * `budget`; a request with len <= budget keeps all.  The kept tokens move in
 * slot order, with their score and position, to the pages of dst_table, which
 * must not be pages that any request still reads; the unused slots of the
 * last block written are zeroed.  A request with a bad length or page id is
 * skipped: kept all -1, new_len = -1, nothing moved.  dst_table needs room for
 * min(budget, max_pages * page_tokens) tokens.
 */
SPEC_API int spec_cache_evict(const spec_cache *cache, const spec_eviction *ev, spec_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
