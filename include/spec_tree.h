/*
 * spec_tree.h -- C ABI of libspecverify: verification of a tree of drafted tokens.
 *
 * A request's packed rows (cu_rows, as in spec_verify.h) are the nodes of a tree:
 * row 0 is its root, the token that the request goes on from, and parent[r] names, by its
 * number within the request, the node that row r's token was drafted after: one before it
 * (0 <= parent < its own number), or -1 for a row that hangs on no other (a slot that the
 * draft left unused).  The root's entry is not looked at; any other value is taken as -1
 * and sets SPEC_STATUS_BAD_TREE.  A chain of drafts is the tree with parent = number - 1.
 *
 * A step appends the nodes' keys and values in the rows' order (spec_cache_append), attends
 * (spec_cache_attend_tree), adjusts the logits, takes a token for every row (row_token of
 * spec_verify_greedy or spec_verify_sample, whose own chain of drafts is not looked at) and
 * follows those tokens through the tree (spec_tree_accept).  Appending the keys and values of
 * path_rows again, from the root's slot on, leaves the accepted path in the cache, where it is a
 * chain (of spec_cache_weights too: the queries and lse of path_rows, with lse = -inf behind the path).
 *
 * Conventions are those of spec_verify.h.
 */
#ifndef SPEC_TREE_H
#define SPEC_TREE_H

#include "spec_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* further device status bits */
#define SPEC_STATUS_BAD_TREE    0x1000u /* a parent that is not before its row: taken as -1        */
#define SPEC_STATUS_BAD_PENALTY 0x2000u /* repetition not finite or <= 0: taken as 1; frequency or
                                           presence not finite: 0; bias offsets malformed: none    */
#define SPEC_STATUS_BAD_MASK    0x4000u /* allowed_row outside [-1, n_allowed): row not masked      */

/* A tree whose rows have got their tokens, and where the accepted path goes. */
typedef struct {
    int32_t B;                 /* requests, >= 1                                              */
    int32_t k_max;             /* at most k_max + 1 rows a request, 0..31                     */
    int32_t R_cap;             /* host-known bound on cu_rows[B]                              */
    const int32_t *cu_rows;    /* [B+1]                                                       */
    const int32_t *row_token;  /* [R_cap] the target's token after each row                   */
    const int32_t *node_token; /* [R_cap] the token that each row was fed (the roots' unread)  */
    const int32_t *parent;     /* [R_cap]                                                     */
    int32_t *accepted_len;     /* [B] accepted nodes below the root, a_b                      */
    int32_t *out_tokens;       /* [B, k_max+1] their tokens, then the target's, then -1       */
    int32_t *next_token;       /* [B] the target's token after the last of them               */
    int32_t *path_rows;        /* [B, k_max+1] or NULL: packed rows of the root and of the
                                  accepted nodes, the last one repeated                       */
    uint32_t *status;          /* [1] or NULL                                                 */
} spec_tree;

/*
 * From the root on, a child whose token is the target's token after the node is
 * accepted (the lowest row where several are) and followed; where no child is,
 * that token is the next one.  For a chain this is the acceptance of the verify calls.  A
 * malformed request (n_b < 1, n_b > k_max + 1, rows outside [0, R_cap]) gets
 * accepted_len = 0 and -1 elsewhere, and sets SPEC_STATUS_BAD_ROWS.  One launch.
 */
SPEC_API int spec_tree_accept(const spec_tree *tree, spec_stream stream);

/* What the logits of a batch's rows are adjusted by. */
typedef struct {
    const void *logits;        /* [R_cap, ld]                                                 */
    int32_t dtype;             /* spec_dtype of logits and out                                */
    int32_t V;                 /* columns, 1 <= V <= ld                                       */
    int64_t ld;
    int32_t B;                 /* requests, >= 1                                              */
    int32_t k_max;             /* at most k_max + 1 rows a request, 0..31                     */
    int32_t R_cap;             /* host-known bound on cu_rows[B]                              */
    const int32_t *cu_rows;    /* [B+1]                                                       */
    const int32_t *history;    /* [B, history_ld] or NULL: each request's tokens so far (the
                                  root's token among them); ids outside [0, V) count nowhere  */
    int64_t history_ld;
    int32_t history_cap;       /* columns of history, at most 2^28 - 64                        */
    const int32_t *n_tokens;   /* [B] how many there are, 0..history_cap                      */
    const int32_t *n_prompt;   /* [B] or NULL (0): how many of them are the prompt's          */
    const float *repetition;   /* [B] or NULL (1): finite, > 0                                */
    const float *frequency;    /* [B] or NULL (0)                                             */
    const float *presence;     /* [B] or NULL (0)                                             */
    const int32_t *node_token; /* [R_cap] or NULL: the token that each row was fed            */
    const int32_t *parent;     /* [R_cap] or NULL: a chain                                    */
    const int32_t *bias_cu;    /* [B+1] or NULL: request b's biases are bias_cu[b] ..         */
    const int32_t *bias_ids;   /* [n_bias] columns, in any order, repeated ones added up      */
    const float *bias_values;  /* [n_bias] finite, or -inf                                    */
    int32_t n_bias;
    const uint32_t *allowed;   /* [n_allowed, allowed_ld] or NULL: bit v % 32 of word v / 32
                                  says whether column v is allowed                            */
    int64_t allowed_ld;        /* words, >= ceil(V / 32)                                      */
    int32_t n_allowed;
    const int32_t *allowed_row;/* [R_cap] or NULL (= row): the mask of each row, -1: none      */
    uint32_t *status;          /* [1] or NULL                                                 */
} spec_logit_rules;

/*
 * For every row r of request b and column v, in fp32:
 *   z = logits[r][v];
 *   if v is among the request's tokens or on the row's path:
 *       z = z > 0 ? z / repetition : z * repetition;
 *   z -= frequency * c + presence * (c > 0), c = how often v is among the generated tokens
 *       (those from n_prompt on) and on the path;
 *   z += the request's biases of v;
 *   z = -inf where the row's mask has bit v clear;
 * rounded once to out's type.  A row's path are the tokens of its ancestors below the
 * root and its own (none at the root, nor at a row that hangs on no other): the drafts that the row's
 * distribution comes after.  With node_token NULL there is none.  out [R_cap, out_ld], out_ld >= V, can be
 * logits itself (with out_ld = ld), and must not overlap it otherwise.  A row whose mask
 * allows nothing comes out as -inf alone.  Rows >= cu_rows[B], and those of a malformed
 * request (n_b < 0, n_b > k_max + 1, rows outside [0, R_cap]: SPEC_STATUS_BAD_ROWS), are not
 * written; an n_tokens out of range counts as 0 (SPEC_STATUS_BAD_LENGTH).
 * One launch: the rows are copied and masked in one pass (in place only those with a mask), and the
 * columns that have a token's count or a bias are read and written once more.
 */
SPEC_API int spec_adjust_logits(const spec_logit_rules *rules, void *out, int64_t out_ld,
                                spec_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_TREE_H */
