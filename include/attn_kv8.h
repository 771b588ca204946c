/*
 * attn_kv8.h - C ABI of the 8-bit paged K/V cache of the B200 (sm_100a) masked attention library.
 *
 * Serving keeps the keys and values of running requests in pages. This header declares a
 * cache that holds them as e4m3 codes with one scale per page and KV head, and the
 * calls around it, in the order of a serving step:
 *   attn_page_tables()  page tables, slot maps and positions from request lengths, on the GPU
 *   attn_kv8_append()   quantise the step's new keys and values into their pages
 *   attn_kv8_fwd()      attention of a few query tokens per request over the cache
 *   attn_kv8_select()   pages that a cheap score selects for each query token; attn_kv8_fwd()
 *                       then attends to those only
 *   attn_kv8_gather()   a request's pages as contiguous bf16 K/V: long query chunks run
 *                       attn_masked_fwd() (any mask of attn.h) on them
 * Lengths, offsets, tables and slots are DEVICE arrays and every call only enqueues work on
 * its stream (nothing is allocated, copied to the host or waited for), so a whole step can be
 * captured into a CUDA graph and replayed while the lengths grow. attn_kv8_plan() is the
 * exception: it allocates the workspace of attn_kv8_fwd().
 *
 * Coordinates as in attn.h: the query tokens of a request are the last of its kv_len tokens,
 * token i of n sits at position kv_len - n + i.
 *
 * Device data is not trusted with memory: lengths are clamped to the table's capacity, query
 * offsets to the token count, and pages outside [0, num_pages) are read as zeros (attention,
 * gather), never selected before any other page, and never written.
 */
#ifndef MASKED_ATTN_B200_ATTN_KV8_H
#define MASKED_ATTN_B200_ATTN_KV8_H

#include <stdint.h>

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache. All pointers are DEVICE pointers, 16-byte aligned (k_scale, v_scale: 4-byte).
 * The block of one page and head is contiguous, so it is read in whole lines whatever hkv is.
 * The value of a code is code * scale, code one of the finite e4m3 values (max 448). A NaN is kept
 * in the scale: a page and head whose scale is NaN read as NaN. The codes 0x7F and 0xFF are
 * never written by attn_kv8_append(); what a call makes of one in a token's place is undefined,
 * bytes in places that no token holds are never used. */
typedef struct {
  void* k;              /* e4m3 [num_pages][hkv][page_size][head_dim] */
  void* v;              /* the same */
  float* k_scale;       /* fp32 [num_pages][hkv], >= 0 or NaN */
  float* v_scale;       /* the same */
  int8_t* k_bounds;     /* int8 [num_pages][hkv][2][head_dim]: per channel the largest (row 0) and the
                           smallest (row 1) K code of the page in steps of 4 codes, rounded
                           outwards (up / down). Written by attn_kv8_append(), read by
                           attn_kv8_select(); NULL when pages are never selected. */
  int32_t num_pages;    /* num_pages * page_size < 2^31 */
  int32_t page_size;    /* 16, 32, 64 or 128 */
  int32_t hkv;          /* KV heads, 1 .. 65535 */
  int32_t head_dim;     /* 64, 128 or 256 */
} attn_kv8_cache_t;

/* Page tables and slot maps of one scheduling step (all arrays DEVICE int32). The free pages
 * are a ring: entries head, head + 1, ... head + count - 1 (modulo num_pages) of free_pages
 * hold the numbers of the free pages; free_state = {head, count, ...}. Request b goes
 * from old_lens[b] to new_lens[b] tokens; L tokens hold ceil(L / page_size) pages.
 *   new > old   the request's next table entries are taken from the ring's head, requests
 *               in order and their pages in order; the tokens old .. new - 1 get slots
 *   new < old   (finished: new = 0; rejected draft tokens) the pages past the new length go to
 *               the ring's tail in the same order; its table entries stay as they were
 * Pages given back in a call are not taken again by the same call. A page belongs to one request: pages are not
 * counted, and one in the rows of two requests (a shared prefix) would go to the ring twice, without a status.
 * Nobody grows (kv_lens = min(old, new), no slots) when the step cannot be done: status 2, a
 * new length is negative or above max_pages_per_seq * page_size (that request stays at its old
 * length); else 3, more new tokens than max_tokens; else 1, too few free pages. Requests that
 * shrink do so all the same, so that a retry can succeed.
 * The call is a function of its inputs: outputs go to buffers of their own (next_state must not
 * be free_state, kv_lens neither old_lens nor new_lens); the table entries it writes and the
 * ring entries it writes are never ones it reads, so a repeated call gives the same result. */
typedef struct {
  int32_t batch;              /* requests, 0 .. 16384 */
  int32_t max_pages_per_seq;  /* row length of page_table, >= 1 */
  int32_t num_pages;          /* entries of free_pages, >= 1 */
  int32_t page_size;          /* 16, 32, 64 or 128 */
  int32_t max_tokens;         /* entries of slots and positions, >= 0 */
  int32_t* page_table;        /* [batch][max_pages_per_seq], updated */
  const int32_t* old_lens;    /* [batch] */
  const int32_t* new_lens;    /* [batch] */
  int32_t* free_pages;        /* [num_pages], updated */
  const int32_t* free_state;  /* [4]: head, count; the others are not read */
  int32_t* next_state;        /* [4]: head, count, status (0 done; 1, 2, 3 above), pages that were missing */
  int32_t* kv_lens;           /* [batch]: the lengths after the step */
  int32_t* cu_seqlens_q;      /* [batch + 1]: offsets of the requests' new tokens */
  int32_t* slots;             /* [max_tokens]: page * page_size + place of each new token, -1 past the last */
  int32_t* positions;         /* [max_tokens]: the token's position in its request, -1 past the last; or NULL */
} attn_page_tables_t;

/* Errors: INVALID_ARG (null pointer, size out of range, an output that is an input), UNSUPPORTED
 * (page_size, batch > 16384), CUDA. */
attn_status_t attn_page_tables(const attn_page_tables_t* tables, attn_stream_t stream);

/* Quantise num_tokens new keys and values into the cache. k_new, v_new: DEVICE bf16 rows of
 * [hkv][head_dim], k_stride / v_stride elements from token to token (>= hkv * head_dim,
 * multiples of 8: views of a fused projection work), 16-byte aligned. slots: DEVICE int32
 * [num_tokens], as attn_page_tables() writes them; a slot outside [0, num_pages * page_size) skips
 * its token. The tokens of one page must follow one another (skipped ones aside) in ascending
 * places, and no page may be written by two requests (else the page's content is undefined).
 * Per page and head, with amax the largest finite |x| of its new tokens:
 *     scale = max(scale before, 2^e), e >= -126 the least with amax <= 448 * 2^e,
 * (a page whose place 0 is among the tokens is new: its scale before counts as 0);
 *     code = x / scale rounded to nearest even, infinities to +-448,
 * and if the scale grew, the codes before become code * before / scale, rounded likewise
 * (exact for powers of two, but for subnormal codes). k_bounds is kept up in the same way.
 * A NaN among the new values makes the scale NaN until place 0 of the page is written again;
 * other pages, heads and (K or V) are not touched by it.
 * Errors: INVALID_ARG (also: k and v, or their scales, overlap), UNSUPPORTED (page_size, head_dim), CUDA. */
attn_status_t attn_kv8_append(const attn_kv8_cache_t* cache, const void* k_new, int64_t k_stride, const void* v_new,
                              int64_t v_stride, const int32_t* slots, int32_t num_tokens, attn_stream_t stream);

/* The cached keys and values of `batch` requests as bf16 rows: row cu_seqlens_k[b] + j of
 * k_out, v_out (bf16 [total_k][hkv][head_dim], 16-byte aligned) is token j of request b. Values
 * code * scale are rounded to bf16 (exact for power-of-two scales, as attn_kv8_append() writes).
 * cu_seqlens_k: DEVICE int32 [batch + 1], non-decreasing from 0; rows from cu_seqlens_k[batch] on
 * are left as they were. page_table: DEVICE int32 [batch][max_pages_per_seq]; tokens past its
 * max_pages_per_seq pages are zeros, as those of pages outside the cache.
 * Errors: INVALID_ARG (also: k_out and v_out overlap), UNSUPPORTED (page_size, head_dim), CUDA. */
attn_status_t attn_kv8_gather(const attn_kv8_cache_t* cache, const int32_t* page_table, int32_t max_pages_per_seq,
                              const int32_t* cu_seqlens_k, int32_t batch, int64_t total_k, void* k_out, void* v_out,
                              attn_stream_t stream);

typedef struct attn_kv8_plan attn_kv8_plan_t; /* opaque */

typedef struct {
  int32_t hq, hkv;      /* query / KV heads, hq % hkv == 0 */
  int32_t head_dim;     /* 64, 128 or 256 */
  int32_t page_size;    /* 16, 32, 64 or 128 */
  float scale;          /* softmax scale; <= 0 selects 1/sqrt(head_dim) */
  int32_t mask;         /* ATTN_MASK_FULL, ATTN_MASK_CAUSAL or ATTN_MASK_SLIDING_WINDOW */
  int32_t window;       /* SLIDING_WINDOW: >= 1 */
  int32_t max_q_len;    /* most query tokens per request that are common (>= 1): picks the kernel's
                           row tile; more tokens are computed too, only less efficiently */
} attn_kv8_problem_t;

/* Make a plan for the current device: the kernel's shape and a workspace for the partial
 * results of requests whose keys several CTAs share (at most 40 MiB). Calls on one plan must be
 * ordered one after another (one stream, or events); streams that overlap need a plan each. A captured
 * graph reads the plan's workspace at every replay: destroy the plan after the graphs that hold its calls.
 * Errors: INVALID_ARG, UNSUPPORTED, OOM, CUDA. */
attn_status_t attn_kv8_plan(const attn_kv8_problem_t* problem, attn_kv8_plan_t** out_plan);
attn_status_t attn_kv8_plan_destroy(attn_kv8_plan_t* plan);

/* The query tokens of one call (pointers are DEVICE pointers). */
typedef struct {
  const void* q;                /* bf16 rows of [hq][head_dim], q_stride elements from token to token, 16-byte aligned */
  int64_t q_stride;             /* >= hq * head_dim, a multiple of 8 */
  int32_t batch;                /* requests */
  int32_t total_q;              /* rows of q, out and lse */
  const int32_t* cu_seqlens_q;  /* int32 [batch + 1], non-decreasing from 0; NULL: one token each (total_q == batch).
                                   Rows from cu_seqlens_q[batch] on are left as they were. */
  const int32_t* page_table;    /* int32 [batch][max_pages_per_seq] */
  int32_t max_pages_per_seq;
  const int32_t* kv_lens;       /* int32 [batch], the query tokens included */
} attn_kv8_batch_t;

/* out[t, h] = softmax_j(scale * q[t, h] . K_j + mask) . V_j and lse (natural log, scale included) over
 * the cached tokens; rows that see no key get out = 0, lse = -inf. out: bf16
 * [total_q][hq][head_dim], 16-byte aligned; lse: fp32 [total_q][hq] or NULL. With `selected` (int32
 * [total_q][hkv][n_selected], as attn_kv8_select() writes it) token t of KV head h sees only keys of the listed
 * pages (numbers of page_table columns; the first min(n_selected, pages it sees) entries are
 * read, a negative or too large one sees nothing; a page listed twice counts twice); the plan's
 * mask applies within them. Products are exact and sums fp32 (q values below 2^-31 of their row's
 * largest, or below 2^-117, lose bits); P is rounded to fp16, by 2^-11 of the largest P of its 16 keys at most, for keys up to
 * 65 nats below the row's maximum. Results do not depend on timing (partial results are
 * joined in a fixed order).
 * Errors: INVALID_ARG (also: another device is current than the plan's, a cache of another shape
 * than the plan's, out overlaps q or lse), CUDA. */
attn_status_t attn_kv8_fwd(const attn_kv8_plan_t* plan, const attn_kv8_cache_t* cache, const attn_kv8_batch_t* batch,
                           const int32_t* selected, int32_t n_selected, void* out, float* lse, attn_stream_t stream);

/* For every query token t and KV head h: the n_selected pages with the highest scores, in
 * ascending order, -1 past the last, into selected (int32 [total_q][hkv][n_selected]). A token at
 * position p sees the pages 0 .. p / page_size. The first `sink` and the last `recent` of them are always
 * selected. The score bounds the largest logit of the page from above (up to the rounding of q): with
 * e the least integer >= -126 such that |q[t, a, :]| <= 127 * 2^e (finite values), qi = q * 2^-e
 * rounded to nearest even (infinities +-127, NaN 0), over the query heads a of h,
 *     score = 4 * k_scale * max_a 2^e sum_c (qi[c] > 0 ? qi[c] * bounds[0][c] : qi[c] * bounds[1][c]),
 * exact integers below 2^24, so equal inputs select equal pages; ties go to the lower
 * page, and a page whose scale is NaN has the largest finite score. scores (fp32 [total_q][hkv][max_pages_per_seq]) receives the scores of the pages a token
 * sees; its other entries are left as they were. The plan's mask must be CAUSAL (or FULL: each
 * token then sees all kv_len tokens). 0 <= sink, 1 <= recent, sink + recent <= n_selected.
 * Errors: INVALID_ARG (also: scores and selected overlap), UNSUPPORTED (a SLIDING_WINDOW plan, more than 64 query
 * heads per KV head), CUDA. */
attn_status_t attn_kv8_select(const attn_kv8_plan_t* plan, const attn_kv8_cache_t* cache, const attn_kv8_batch_t* batch,
                              int32_t sink, int32_t recent, float* scores, int32_t* selected, int32_t n_selected,
                              attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MASKED_ATTN_B200_ATTN_KV8_H */
