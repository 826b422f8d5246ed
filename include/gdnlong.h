/*
 * gdnlong: long contexts in the paged cache of gdnhybrid.h, on NVIDIA GB300
 * (sm_103a).  Requests that begin alike read their common pages once, and
 * tokens that few rows attend to leave the cache.  C ABI, in the same library
 * and in the same manner: every buffer belongs to the caller, nothing is
 * allocated, nothing synchronises, every call is asynchronous on `stream` and can
 * be captured in a CUDA graph; return codes are gdnspec.h's GDN_OK and
 * GDN_ERR_*; values only the device sees are skipped and OR a bit into *status
 * (which may be NULL).  Kernels are chained by programmatic dependent launch as
 * gdnhybrid.h states.  Pools, slots, tables, rows and lengths are gdnhybrid.h's.
 * Two calls that share a work buffer, or write the same slots, must not run at
 * the same time.
 *
 * Eviction, a step at a time:
 *   gdn_shared_attention  each attention layer: o, and each row's lse
 *   gdn_attn_weight       each layer: what every cached token got of the rows' attention
 *   gdn_evict_select      when a request passes its budget: the lightest tokens leave
 *   gdn_kv_move           each layer: K and V of the tokens that close the gaps
 * and the next gdn_page_map, given the shorter lengths, takes the pages back.  A
 * request's tokens then lie in the cache in no order of time: attention does not
 * ask for one, as rows see every cached token, and positions are in K.  A token's
 * index in the cache (page of its table row and place in it) and its position in
 * the text differ from the first eviction on: the text's length is the cache's
 * plus the tokens that left.
 *
 * Pages of a shared prefix.  gdn_page_map knows none: to it the first held[b] entries
 * of a table row are request b's alone, and go back to the ring when b's lengths
 * need them no more.  So while several requests hold a prefix of L tokens, W = L /
 * page_size whole pages, none of their lengths may fall below W * page_size in a
 * call, or those pages are in the ring while others read them, once for each
 * request that ends, and later in two requests.
 *   A request joins: the caller writes the W pages into its table row, held[b] = W,
 *     ctx_len[b] = L.  Where L is no multiple of page_size the next gdn_page_map
 *     takes a page of its own for the rest, and gdn_kv_move brings the rest's tokens
 *     there from a request that has them, before attention reads them.  (Where pages
 *     did not suffice held_out[b] is still W, and the table has no such page: nothing
 *     may be moved, ctx_len[b] goes back to W * page_size for the step's other calls,
 *     and the request joins in a later step.)
 *   It lives: first[b] of gdn_attn_weight and pinned[b] of gdn_evict_select are L or
 *     more, so that no call writes what others read.
 *   It ends, and others hold the prefix: a gdn_page_map with ctx_len[b] = W *
 *     page_size, n_rows[b] = 0 takes the pages behind it; before the next one
 *     held[b] = ctx_len[b] = 0.
 *   The last one ends as any request does, with ctx_len[b] = n_rows[b] = 0.
 */
#ifndef GDNLONG_H
#define GDNLONG_H

#include "gdnhybrid.h"

#ifdef __cplusplus
extern "C" {
#endif

/* status bits beside gdnspec.h's and gdnhybrid.h's */
enum {
  GDN_STATUS_MOVES_FULL = 1024, /* an eviction needs more moves than its lists hold: request left as it was */
  GDN_STATUS_BAD_GROUP = 2048   /* group_start does not rise within [0, B]: no prefix is shared in this call */
};

/* ---- attention over shared prefixes -----------------------------------------
 * o as gdn_paged_attention computes it, to the rounding of sums taken in another
 * order, and lse[r][i] = ln sum_j exp(scale * (q[r][i] . K[j])) over the keys row
 * r sees.  Requests group_start[g] .. group_start[g+1]-1 form group g, and are
 * taken to hold the same first prefix_len[g] tokens: the rows of all of them that
 * have at least so many cached tokens meet those keys together, read once, through
 * the table row of the first of them that has rows.  (Pages before the prefix's
 * end are usually the same pages; where a prefix ends inside a page, each
 * request's table has its own copy of that page.)  Requests outside every group,
 * with fewer cached tokens than their group's prefix, or whose rows times
 * H_q/H_kv fill a tile (128 in bf16, 32 in f32) read everything through their own
 * table row, as do all where prefix_len is not positive, and where by an estimate
 * from the lengths reading together saves less than joining the two parts of a row
 * costs.  Which way a request goes changes o and lse by the rounding of sums alone.
 * A call in which nothing is shared takes 8 to 14 % longer than
 * gdn_paged_attention, small ones 3 us: that one serves better where neither
 * prefixes nor lse are wanted.
 *
 *   attn         the call as gdn_paged_attention takes it; attn.work:
 *                gdn_shared_attention_work_bytes(args) bytes, 16-byte aligned
 *   group_start  [n_groups + 1] int32, prefix_len [n_groups] int32 (both may be
 *                NULL where n_groups is 0)
 *   lse          [n_q_rows] rows of H_q fp32, lse_row_stride elements apart (>= H_q);
 *                NULL: not wanted.  Rows of no request are not written
 *
 * Arithmetic, waits and limits are gdn_paged_attention's; lse is 32-bit
 * throughout.  Supported beside that: B <= 4096, n_groups <= 512. */
typedef struct gdn_shared_attn_args {
  gdn_paged_attn_args attn;
  int32_t n_groups;
  int32_t reserved; /* 0 */
  const int32_t* group_start;
  const int32_t* prefix_len;
  float* lse;
  int64_t lse_row_stride;
} gdn_shared_attn_args;
GDN_API int gdn_shared_attention(const gdn_shared_attn_args* args, void* stream);

/* Bytes of attn.work: a function of B, d, in_dtype, H_q, H_kv and n_q_rows alone
 * (not of the groups, which may change from call to call), and no smaller for a
 * larger B or n_q_rows.  Beside gdn_paged_attention's, 2 * H_q * (4 d + 16) bytes
 * for each row that can take part in a prefix: n_q_rows, but at most B times the
 * rows of a request that do not fill a tile.  0 if the sizes are unsupported. */
GDN_API size_t gdn_shared_attention_work_bytes(const gdn_shared_attn_args* args);

/* ---- attention weight of cached tokens ---------------------------------------
 * For every active request b and cache index j, first[b] <= j < ctx_len[b] +
 * n_rows[b], with s the slot of j:
 *   got = sum over rows t with ctx_len[b] + t >= j, over query heads i, of
 *         exp(scale * (q[t][i] . K[j][i / (H_q/H_kv)]) - lse[t][i])
 *   weight[s] = keep * weight[s] + got
 * Each row and head hands out a weight of 1 in all, so that after a request's
 * first step its weights sum to n_rows * H_q.  With `fresh`, tokens of the step
 * itself (j >= ctx_len[b]) start anew, whatever their slot held: weight[s] = got;
 * and born[s] = position[b] + j - ctx_len[b] for all of them.  A step's layers
 * share one array: the first call takes fresh and keep, the others neither (0 and 1).
 * Rows that do not count (drafts turned down) are left out by a smaller n_rows.
 * first[b] keeps a shared prefix's tokens, and others that never leave, out of
 * it: two requests of a call must not hold the same slot at or behind their first.
 *
 *   q, k_cache, block_table, ctx_len, n_rows, row_start, R  as gdn_paged_attention's
 *   lse      [n_q_rows] rows of H_q fp32 (gdn_shared_attention)
 *   first    [B] int32 (NULL: 0); position [B] int32 (NULL: ctx_len)
 *   weight   [n_pages * page_size] fp32, by slot
 *   born     [n_pages * page_size] int32, by slot (may be NULL)
 *   work     gdn_attn_weight_work_bytes(args) bytes, 16-byte aligned; contents on
 *            entry do not matter
 * Arithmetic: products of the inputs' type with 32-bit sums, exponentials and
 * weights in 32 bits, added in an order that depends on the lengths alone.  The
 * same inputs give the same bits on every call.  Supported sizes, alignments and skipped
 * requests are gdn_paged_attention's.  q's strides are not negative, and for
 * GDN_DTYPE_BF16 below 2^39 elements, as the pool's.  A page outside the pool
 * (GDN_STATUS_BAD_PAGE) takes no weight.  A negative first counts as 0. */
typedef struct gdn_attn_weight_args {
  int32_t B, R;
  int32_t H_q, H_kv, d;
  int32_t page_size, n_pages;
  int32_t max_pages, table_stride;
  int32_t n_q_rows;
  int32_t in_dtype;
  int32_t fresh; /* 0 or 1 */
  float scale;   /* as gdn_paged_attn_args */
  float keep;    /* finite */
  const void* q;
  int64_t q_row_stride, q_head_stride;
  const void* k_cache;
  int64_t k_page_stride, k_head_stride, k_token_stride;
  const float* lse;
  int64_t lse_row_stride;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* n_rows;
  const int32_t* row_start;
  const int32_t* first;
  const int32_t* position;
  float* weight;
  int32_t* born;
  void* work;
  int32_t* status;
} gdn_attn_weight_args;
GDN_API int gdn_attn_weight(const gdn_attn_weight_args* args, void* stream);

/* Bytes of `work`: a function of d and in_dtype alone.  0 if the sizes are
 * unsupported. */
GDN_API size_t gdn_attn_weight_work_bytes(const gdn_attn_weight_args* args);

/* ---- which tokens leave ---------------------------------------------------------
 * For every request b, of its ctx_len[b] tokens:
 *   may leave   index j >= pinned[b], and born[slot of j] < keep_from[b]
 *   leave       as many as ctx_len[b] is over max(budget[b], 0), but no more than may:
 *               the lightest first, of equal weights the last index first; NaN
 *               weighs as much as -infinity
 *   ctx_out[b] = K, the tokens that stay.  The i-th index below K that a token left
 *   (rising) takes the i-th token that stays at or above K: move_to[b][i] and
 *   move_from[b][i] are their slots, n_moves[b] their number, and weight and born
 *   move at once.  No slot is in both lists, so that K and V can move in any order.
 *   Entries behind n_moves[b] are not written.
 * No order of tokens is kept; see above.
 *
 *   ctx_len, budget [B] int32; pinned [B] (NULL: 0), keep_from [B] (NULL, or no
 *   born: no such bound)
 *   block_table [B][table_stride], entries of the request's tokens
 *   weight [n_pages * page_size] fp32 and born int32 (may be NULL), by slot: in/out
 *   ctx_out [B] int32: may be ctx_len itself
 *   move_from, move_to [B][max_moves] int32; n_moves [B] int32
 *
 * A request is left as it is (ctx_out = ctx_len, no moves) where ctx_len is
 * negative or beyond the table row (GDN_STATUS_BAD_LENGTH), a page of its tokens
 * lies outside the pool (GDN_STATUS_BAD_PAGE), or it needs more than max_moves
 * moves (GDN_STATUS_MOVES_FULL).  Two requests must not hold the same slot at or
 * behind their pinned.
 * Time: a table row that can hold more than 16384 tokens (max_pages * page_size)
 * gives every request eight blocks in place of one, whatever its length.  Where
 * requests are many and short, pass the pages that they may have, not the row's
 * width (128 requests of 1000 to 8000 tokens: 17 us, and 146 with max_pages for
 * 131072 tokens).
 * Supported: B <= 65535, page_size >= 1, n_pages * page_size < 2^31,
 * B * max_moves < 2^31. */
typedef struct gdn_evict_args {
  int32_t B;
  int32_t page_size, n_pages;
  int32_t max_pages, table_stride;
  int32_t max_moves;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* budget;
  const int32_t* pinned;
  const int32_t* keep_from;
  float* weight;
  int32_t* born;
  int32_t* ctx_out;
  int32_t* n_moves;
  int32_t* move_from;
  int32_t* move_to;
  int32_t* status;
} gdn_evict_args;
GDN_API int gdn_evict_select(const gdn_evict_args* args, void* stream);

/* ---- K and V of the moved tokens --------------------------------------------------
 * For every request b, i < n_moves[b] and head: the d elements of K and V at slot
 * move_from[b][i] to slot move_to[b][i].  No slot may be in both lists, or twice in
 * move_to.  A move from or to a slot outside the pool is skipped
 * (GDN_STATUS_BAD_PAGE), a request whose n_moves is outside [0, max_moves] too
 * (GDN_STATUS_BAD_LENGTH).  Pointers and strides are multiples of 16 bytes, and
 * so is d.  Supported: B <= 65535, B * max_moves < 2^31, n_pages * page_size < 2^31.
 * Time: blocks are launched for max_moves moves of every request, and those without
 * one end at once: lists no longer than an eviction can need cost least (10 moves of
 * each of 16 requests, 8 heads of 128 in bf16: lists of 64 2.1 us, of 4096 17). */
typedef struct gdn_kv_move_args {
  int32_t B, max_moves;
  int32_t H_kv, d;
  int32_t page_size, n_pages;
  int32_t in_dtype;
  int32_t reserved; /* 0 */
  const int32_t* move_from;
  const int32_t* move_to;
  const int32_t* n_moves;
  void* k_cache;
  void* v_cache;
  int64_t k_page_stride, k_head_stride, k_token_stride;
  int64_t v_page_stride, v_head_stride, v_token_stride;
  int32_t* status;
} gdn_kv_move_args;
GDN_API int gdn_kv_move(const gdn_kv_move_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GDNLONG_H */
