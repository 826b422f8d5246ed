/*
 * gdnhybrid: the rest of a Qwen3.5-style hybrid's verify step beside its
 * GatedDeltaNet layers (gdnspec.h), on NVIDIA GB300 (sm_103a): where the
 * step's new tokens go in a paged cache, the append of their K and V rows, the
 * full attention of a request's new tokens over its pages, and the acceptance
 * of drafts against sampled target tokens.  C ABI, in the same library and in
 * the same manner: every buffer belongs to the caller, nothing is allocated,
 * nothing synchronises, every call is asynchronous on `stream` and can be
 * captured in a CUDA graph; return codes are gdnspec.h's GDN_OK and
 * GDN_ERR_*; values only the device sees are skipped and OR a bit into
 * *status (which may be NULL).  Kernels of one call, and of calls that follow
 * each other, are chained by programmatic dependent launch: each waits for
 * what ran before it on the stream before it reads or writes anything, and a
 * kernel launched behind a call with programmatic stream serialization must
 * wait too (griddepcontrol.wait) before it uses the call's outputs.
 *
 * The paged cache.  K and V pools of n_pages pages, each page holding
 * page_size consecutive tokens of one request for all H_kv heads.  A pool is
 * addressed as base + page*page_stride + head*head_stride + token*token_stride
 * (strides in elements, not negative; the d elements of a token and head are
 * contiguous), so head-major [pages][H_kv][P][d], token-major
 * [pages][P][H_kv][d] and pools that interleave K and V are all the same call.
 * block_table[b][i] is the page of request b's tokens i*P .. i*P+P-1; a slot is
 * page*P + token.
 *
 * Rows.  A step's new tokens are rows of q, k, v and o.  Request b has
 * n_rows[b] of them (0 = inactive) behind ctx_len[b] tokens that the cache
 * holds; its row t is the token at position ctx_len[b] + t and lies at row
 * row_start[b] + t.  With R > 0 rows are padded, R to a request (row_start[b] =
 * b*R, as x and o of gdnspec.h); with R = 0 they are packed.
 */
#ifndef GDNHYBRID_H
#define GDNHYBRID_H

#include "gdnspec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* status bits beside gdnspec.h's */
enum {
  GDN_STATUS_NO_PAGES = 32,    /* the free pages did not suffice: request not served     */
  GDN_STATUS_TABLE_FULL = 64,  /* a request needs more pages than its table row holds,
                                  or holds a count outside [0, max_pages] or more pages
                                  than there are: not served                             */
  GDN_STATUS_BAD_PAGE = 128,   /* a page or slot outside the pool: skipped, or read as
                                  zeros (gdn_paged_attention)                            */
  GDN_STATUS_BAD_LENGTH = 256, /* a negative ctx_len, or more tokens than the table row
                                  or the rows of q hold: request skipped                 */
  GDN_STATUS_ROWS_FULL = 512   /* packed rows beyond the row arrays: the request, and any
                                  behind it, gets no rows this step                      */
};

/* ---- page map: tables, slots and positions from request lengths -----------
 * One call per step.  Request b needs need = ceil((ctx_len[b] + n_rows[b]) / P)
 * pages.  Where it holds fewer (held_in[b]) it takes the missing ones off the
 * head of the free ring; where it holds more (drafts turned down, or a
 * finished request with ctx_len = n_rows = 0) it gives the surplus back at the
 * ring's tail; both in request order, so the same inputs give the same pages.
 * Requests are served in order while the cumulative demand fits the free
 * pages: one whose demand does not fit keeps what it holds, gets no rows
 * (rows_out[b] = 0, GDN_STATUS_NO_PAGES), and its demand still counts for the
 * ones behind it; a request that needs no page is always served.  Pages given
 * back in a call are free from the next call on.
 *
 *   ctx_len, n_rows, held_in  [B] int32
 *   free_ring  [n_pages] int32  in/out: free pages at ring positions head .. head+free-1 (mod n_pages)
 *   free_in    [2] int32        head and number of free pages before the call
 *   block_table[B][table_stride] int32 in/out: entries held_in[b]..need-1 are written, none is cleared
 *   held_out   [B] int32        pages held after the call
 *   free_out   [2] int32        the ring's head and free pages after the call
 *   rows_out   [B] int32        rows served: n_rows[b], or 0 (not served)
 *   row_start  [B+1] int32      b*R, or packed the prefix of the rows that pages sufficed for; [B] = all of them.
 *              Rows beyond the row arrays (GDN_STATUS_ROWS_FULL) count here although rows_out does not have them
 *   slot_map, positions [n_slot_rows] int32   per row; -1 for rows of no token.  Padded: B*R of them;
 *              without either n_slot_rows does not matter
 *
 * held_out and rows_out must not overlap ctx_len, n_rows, held_in or free_in,
 * nor free_out free_in: a step's blocks read the old counts while they write the
 * new ones (keep two of held and free and alternate; GDN_ERR_INVALID_ARG
 * otherwise).  A negative ctx_len or n_rows, or n_rows > R
 * when padded, leaves the request's pages as they are, rows_out 0
 * (GDN_STATUS_BAD_LENGTH, GDN_STATUS_BAD_NROWS).  Any output but
 * block_table, held_out, free_out, rows_out may be NULL.  With B = 0 the counts
 * go from free_in to free_out and rows are written as rows of no token; without
 * both of the two such a call does nothing.
 * Supported: B <= 4096, page_size >= 1, n_pages*page_size < 2^31. */
typedef struct gdn_page_map_args {
  int32_t B, R;
  int32_t page_size, n_pages;
  int32_t max_pages;    /* usable entries of a table row   */
  int32_t table_stride; /* >= max_pages                    */
  int32_t n_slot_rows;  /* rows of slot_map and positions  */
  int32_t reserved;     /* 0 */
  const int32_t* ctx_len;
  const int32_t* n_rows;
  const int32_t* held_in;
  int32_t* free_ring;
  const int32_t* free_in;
  int32_t* block_table;
  int32_t* held_out;
  int32_t* free_out;
  int32_t* rows_out;
  int32_t* row_start;
  int32_t* slot_map;
  int32_t* positions;
  int32_t* status;
} gdn_page_map_args;
GDN_API int gdn_page_map(const gdn_page_map_args* args, void* stream);

/* ---- append: K and V rows of the new tokens into their slots ---------------
 * For every row r with slot_map[r] >= 0 and every head: the d elements of
 * k[r][h] and v[r][h] to the pools at that slot.  A negative slot is a row of
 * no token; one beyond the pool is skipped (GDN_STATUS_BAD_PAGE).  Two rows
 * must not name the same slot.  k and v may be slices of a fused projection's
 * rows (strides in elements).  Pointers and strides are multiples of 16 bytes,
 * and so is d. */
typedef struct gdn_kv_append_args {
  int32_t rows, H_kv, d;
  int32_t page_size, n_pages;
  int32_t in_dtype; /* GDN_DTYPE_* of k, v and the pools */
  const void* k;
  const void* v;
  int64_t k_row_stride, k_head_stride, v_row_stride, v_head_stride;
  const int32_t* slot_map; /* [rows] */
  void* k_cache;
  void* v_cache;
  int64_t k_page_stride, k_cache_head_stride, k_token_stride;
  int64_t v_page_stride, v_cache_head_stride, v_token_stride;
  int32_t* status;
} gdn_kv_append_args;
GDN_API int gdn_kv_append(const gdn_kv_append_args* args, void* stream);

/* ---- attention of a request's new tokens over its pages ---------------------
 * For every active request b, row t < n_rows[b] and query head i, with kv head
 * h = i / (H_q / H_kv) and j over positions 0 .. ctx_len[b] + t:
 *   o = sum_j p_j V[j][h] / sum_j p_j,   p_j = exp(scale * (q . K[j][h]) - max)
 * The new tokens' own K and V are read from the cache (append them first).
 * One row and one request, verify rows, and prompt chunks of any length are
 * the same call; lengths are read on the device.  Rows of no request are not
 * written.  Tokens past a request's length (the rest of its last page) may
 * hold anything, NaN included; a V row of the request's own new tokens that is
 * not finite may reach the chunk's earlier rows too.
 *
 *   q, o        [n_q_rows][H_q][d] in_dtype, with row and head strides
 *   block_table [B][table_stride]; entries past a request's tokens are not read
 *   ctx_len, n_rows [B]; row_start [B] (NULL: b*R)
 *   work        gdn_paged_attention_work_bytes(args) bytes, 16-byte aligned:
 *               partial results of rows whose keys are split over several
 *               blocks; contents on entry do not matter
 *
 * Arithmetic.  GDN_DTYPE_F32: 32-bit products and sums throughout.
 * GDN_DTYPE_BF16: products of bf16 with 32-bit sums; the weights p are rounded
 * to bf16 before they meet V (their sum is not); o is rounded once.
 * The same inputs give the same bits on every call.  A kernel never spins
 * without bound: where a staging copy does not land in time, the block that
 * waits for it gives up, GDN_STATUS_TIMEOUT is set, and the o rows it had a part
 * in are undefined.
 *
 * Supported: d in {64, 128, 256}; H_q a multiple of H_kv, H_q/H_kv <= 128;
 * page_size a multiple of 16 up to 1024 (any >= 1 for GDN_DTYPE_F32).
 * q, o, pools and work 16-byte aligned, strides multiples of 16 bytes.
 * A request with a negative ctx_len or with more tokens than max_pages pages,
 * n_rows outside [0, R] (padded), rows outside q, or more than 2^31 - 1024
 * tokens or rows times H_q/H_kv is skipped with its bit. */
typedef struct gdn_paged_attn_args {
  int32_t B, R;
  int32_t H_q, H_kv, d;
  int32_t page_size, n_pages;
  int32_t max_pages, table_stride;
  int32_t n_q_rows;
  int32_t in_dtype;
  float scale; /* finite, and scale * log2(e) too: up to 2.35e38 */
  const void* q;
  int64_t q_row_stride, q_head_stride;
  const void* k_cache;
  int64_t k_page_stride, k_head_stride, k_token_stride;
  const void* v_cache;
  int64_t v_page_stride, v_head_stride, v_token_stride;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* n_rows;
  const int32_t* row_start;
  void* o;
  int64_t o_row_stride, o_head_stride;
  void* work;
  int32_t* status;
} gdn_paged_attn_args;
GDN_API int gdn_paged_attention(const gdn_paged_attn_args* args, void* stream);

/* Bytes of `work`: a function of d and in_dtype alone.  0 if the sizes are
 * unsupported. */
GDN_API size_t gdn_paged_attention_work_bytes(const gdn_paged_attn_args* args);

/* ---- acceptance of drafts against sampled target tokens --------------------
 * gdn_greedy_accept for requests that sample.  For every request b with
 * 0 < n_rows[b] <= R and every verify row t < n_rows[b], with l the row's
 * logits, T, k, p, m the request's temperature, top_k, top_p, min_p and u the
 * row's random number:
 *   weights     W_i = rint(2^31 * w_i), w_i = exp((l_i - max l) * (1 / T)),
 *               where l_i == max l: w_i = 1; NaN logits take no part
 *   top-k       the k first tokens by logit, equal logits by lowest index
 *   top-p       of those, in that order, every token before which the running
 *               W sum is below floor(p * 2^24) / 2^24 of their total; the
 *               first token always
 *   min-p       of those, the tokens with w_i >= min(m, 1)
 *   target      the first token, by index, at which the running W sum of the
 *               kept tokens exceeds floor(u * 2^24) / 2^24 of their total
 *   prob        w_target * 2^31 / (kept total): its probability after all filters
 * Weights are whole numbers, so every sum is exact and the result does not
 * depend on the order of summation.  temperature not above 0: the largest
 * logit (lowest index among equals), prob 1.  A row of NaN gives token 0 with
 * prob 1, as greedy acceptance does.  k <= 0 or >= V, p >= 1 (or NaN), m <= 0
 * (or NaN) switch a filter off; p <= 0 keeps one token; u is clamped to [0, 1).
 * Drafts are accepted as in gdn_greedy_accept: accept_len[b] = the largest a <=
 * n_rows[b]-1 with drafts[b][i] == target[b][i] for all i < a.  Accepting a
 * draft only where the target's own sample equals it leaves the target's
 * distribution unchanged.
 *
 *   logits  [B][R] rows of V, in_dtype, row_stride elements apart (>= V).  Any V
 *           and any stride; rows that start on 16 bytes are read fastest
 *   u       [B][R] fp32 in [0, 1)
 *   temperature, top_k, top_p, min_p [B] fp32, int32, fp32, fp32; each may be NULL (1, off, off, off)
 *   drafts  [B][R-1] int32 (NULL: no accept_len wanted, or R == 1); n_rows [B]
 *   target  [B][R] int32, prob [B][R] fp32 (may be NULL): rows t >= n_rows[b] are not written
 *   accept_len [B] int32 (NULL: not wanted); 0 for inactive requests and for a bad n_rows
 * Supported: V <= GDN_SAMPLE_MAX_V (a row is staged in the shared memory of at
 * most eight blocks), B, R <= 65535. */
typedef struct gdn_sample_args {
  int32_t B, R, V;
  int32_t in_dtype;
  int64_t row_stride;
  const void* logits;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const int32_t* drafts;
  const int32_t* n_rows;
  int32_t* target;
  float* prob;
  int32_t* accept_len;
  int32_t* status;
} gdn_sample_args;
#define GDN_SAMPLE_MAX_V 393216
GDN_API int gdn_sample_accept(const gdn_sample_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GDNHYBRID_H */
