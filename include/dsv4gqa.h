/*
 * dsv4gqa.h - C ABI of the grouped-query cache operators: the write, the
 * one-token attention and the eviction of a paged cache with separate K and V
 * rows.
 *
 * They serve a model with ordinary grouped-query heads (num_kv_heads heads
 * with K and V rows of head_dim values, each shared by num_heads /
 * num_kv_heads query heads) beside the one that dsv4attn.h serves, for
 * instance a separate model that drafts tokens for dsv4_attn_verify.  The
 * DeepSeek-V4 caches, whose 512-wide rows are key and value at once (those of
 * its own draft layer too), stay with the kernels of dsv4attn.h.  These
 * operators have no counterpart on the source pages.
 *
 * The cache (dsv4_gqa_cache)
 *   Slot s of request row r lies on physical page
 *     page = page_table[r * page_table_stride + s / page_size]
 *   and its K row for KV head h starts at byte
 *     page * page_stride + h * head_stride + (s % page_size) * row_stride
 *   of k (the V row at the same offset of v).  Any order of page, head and
 *   row fits (head-major and token-major pages alike); the head_dim values of
 *   a row are contiguous.  A cache of E4M3 rows stands for
 *   code * k_scale[h] (v_scale[h]).
 *
 * dsv4_gqa_store: for i = 0 .. n-1, r = req_rows[i], s = slots[i] and every
 *   KV head h: the K and V rows of token i go to slot s of request row r,
 *   unchanged, or for an E4M3 cache as the e4m3 code nearest to x / scale[h]
 *   (fp32 quotient, ties to even, saturating at +-448; NaN stays NaN).  With
 *   `weights`, weights[r][h][s] becomes 0; with `positions`,
 *   positions[r][h][s] becomes token_positions[i].  When two indices address
 *   the same slot, which of their values each 16-byte piece gets is not
 *   defined.
 *
 * dsv4_gqa_decode: request b (request row r) has n = lens[b] cached rows and
 *   one query row of num_heads heads.  For query head i of KV head
 *   h = i / (num_heads / num_kv_heads), with lo = window ? max(0, n - window)
 *   : 0,
 *     s_j = scale * <q_i, K_j>,  j = lo .. n-1
 *     L   = exp(sink[i]) + sum_j exp(s_j)          (no sink: that term is 0)
 *     out = sum_j exp(s_j) V_j / L       lse = ln L
 *   Scores, softmax statistics and sums are fp32, products of 16-bit values
 *   exact; the weight of a row enters its product with V with an error of at
 *   most 2^-17 of it, or 2^-12 where the cache is E4M3 and out bf16, and 2^-36
 *   of the largest weight (F16 and E4M3 caches).
 *   A request with no rows gets out = 0 and lse = sink[i] (or -inf).  An
 *   infinite value of an attended V row makes its dim of out infinite (NaN
 *   where both signs or a NaN meet), as the sum does; finite bf16 values must
 *   stay below 2^90, where fp32 sums of 2^30 rows cannot overflow.  With
 *   `weights_out`, for j = 0 .. n-1,
 *     weights_out[r][h][j] = decay * weights[r][h][j]
 *                            + sum over the heads i of h of exp(s_j - lse_i)
 *   (the sum is empty for j < lo); entries behind the last row are left as
 *   they were.  Requests of one call that name the same row add up.
 *
 * dsv4_gqa_evict: request b (row r) has n = lens[b] cached rows; where
 *   n > keep, every KV head h keeps `keep` of them: first the rows whose
 *   position is below `first` or at least seq_lens[b] - recent, then those
 *   with the largest weights[r][h][s], equal ones by lower slot (NaN ranks
 *   with -inf).  Kept rows stay in their slots if those lie below `keep`; the
 *   others, in ascending order, take the slots of the evicted rows below
 *   `keep`, in ascending order, so only what has to move moves: K and V row,
 *   weight and position.  lens_out[b] = min(n, keep).  Slots from `keep` on
 *   are left as they were.  After an eviction a slot's number no longer is
 *   its position: `positions` keeps it (NULL: position = slot, as in a cache
 *   that has lost nothing yet), and `window` of dsv4_gqa_decode, which counts
 *   slots, no longer applies.
 *   weights_out / positions_out may be the same array as weights / positions;
 *   where they are others, the surviving entries are copied.  The pages that
 *   hold a request's first `keep` slots must not belong to another request of
 *   the call too.  A request row that the call names twice is evicted for the
 *   first of them; the later ones set DSV4_DEV_ERR_REQ_ROW.
 *
 * Conventions
 *   Memory, streams and errors are those of dsv4attn.h: device memory owned
 *   by the caller, asynchronous on `stream`, nothing allocated, a negative
 *   DSV4_ERR_* before any launch for what the host can check, and for what it
 *   cannot a bit in the error word of dsv4_attn_get_device_error(): a length
 *   below 0 or above max_len is clamped into the range
 *   (DSV4_DEV_ERR_GQA_LENGTH), a request row outside the table counts as a
 *   request without rows (DSV4_DEV_ERR_REQ_ROW; unreported for length 0, so
 *   a padded batch may hold any row there), rows on a page id outside the
 *   pool are skipped (DSV4_DEV_ERR_GQA_PAGE), a stored row that has no place
 *   is skipped (DSV4_DEV_ERR_STORE_ROW).  DSV4_DEV_ERR_TIMEOUT after a decode
 *   call: a wait inside its kernel was given up (a library bug), and what the
 *   call wrote to its outputs is undefined; later calls are not affected.
 *   Every kernel can be captured into a graph.  Before any capture on a device
 *   make one call there of each function, and of dsv4_gqa_decode one for each
 *   cache format, query type and head_dim: it loads every kernel that calls
 *   of these can take, whatever their sizes and optional arguments.
 *   A captured call reads lens, tables and rows anew at every replay.
 *   lens, seq_lens, req_pool_indices: int32 [batch]; req_pool_indices NULL =
 *   request b is row b.
 *   weights (fp32) and positions (int32): [page_table_rows, num_kv_heads,
 *   width], width >= max_len.
 *   max_len: bound on lens; at most page_table_width * page_size and 2^30.  It
 *   sizes launches and workspaces and chooses between them, so give the
 *   smallest that is known: a decode call whose max_len is short takes one
 *   launch, an eviction does where max_len - keep <= 4 (and lens_out is neither
 *   lens nor seq_lens), and the workspace of a decode call with weights has 32
 *   to 256 bytes for each slot up to max_len of each request and KV head.
 *   Limits, beyond which a call returns DSV4_ERR_UNSUPPORTED: batch *
 *   num_kv_heads of an eviction or of a decode call with weights is at most
 *   65535; requests * KV heads * groups of up to 16 query heads of a decode
 *   call is at most 2^30, and times the tiles of max_len slots (at least 16
 *   slots each) less than 2^31.
 *   workspace: device scratch of at least the size that the matching
 *   _workspace_size function gives, 16-byte aligned; need not be initialised
 *   and holds nothing between calls.  Calls that may run at the same time
 *   (graph replays among them) need workspaces of their own.
 */
#ifndef DSV4GQA_H
#define DSV4GQA_H

#include <stddef.h>
#include <stdint.h>

#include "dsv4attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types ---- */
#define DSV4_GQA_BF16  0
#define DSV4_GQA_F16   1
#define DSV4_GQA_E4M3  2   /* cache rows only */

/* ---- device error bits (dsv4_attn_get_device_error) ---- */
#define DSV4_DEV_ERR_GQA_PAGE    0x200u  /* a row on a page id outside the pool */
#define DSV4_DEV_ERR_GQA_LENGTH  0x400u  /* a length outside 0..max_len */

typedef struct dsv4_gqa_cache {
    void*          k;                   /* device, 16-byte aligned */
    void*          v;                   /* device, 16-byte aligned, same strides */
    int64_t        num_pages;
    int64_t        page_stride;         /* bytes, multiples of 16 */
    int64_t        head_stride;
    int64_t        row_stride;
    const int32_t* page_table;          /* device int32 [page_table_rows, page_table_stride] */
    int32_t        page_table_rows;
    int32_t        page_table_stride;
    int32_t        page_table_width;    /* logical pages per request row, <= page_table_stride */
    int32_t        num_kv_heads;        /* 1 .. 256 */
    int32_t        head_dim;            /* 64, 128 or 256 */
    int32_t        page_size;           /* a power of two, 16 .. 1024 */
    int32_t        format;              /* DSV4_GQA_BF16, DSV4_GQA_F16 or DSV4_GQA_E4M3 */
    const float*   k_scale;             /* device fp32 [num_kv_heads], > 0; E4M3 only, NULL = 1 */
    const float*   v_scale;
} dsv4_gqa_cache;

/* k, v: n tokens (at most 2^30) of num_kv_heads rows, type BF16 or F16 (the cache's own type
   unless that is E4M3); strides in elements, multiples of 8; 16-byte aligned.
   weights / positions may be NULL; token_positions int32 [n] goes with
   positions; width as above. */
int dsv4_gqa_store(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                   const void* v, int64_t v_token_stride, int64_t v_head_stride,
                   int32_t type, int32_t n, const int32_t* req_rows, const int32_t* slots,
                   const dsv4_gqa_cache* cache, float* weights, int32_t* positions, int64_t width,
                   const int32_t* token_positions, void* stream);

/* q: batch rows of num_heads * head_dim contiguous values, q_stride elements
   apart (a multiple of 8), type BF16 or F16 (the cache's own type unless that
   is E4M3), 16-byte aligned.  out: the same type, [batch, num_heads, head_dim]
   contiguous, 16-byte aligned.  sink fp32 [num_heads] or NULL; lse fp32
   [batch, num_heads] or NULL.  num_heads is a multiple of num_kv_heads, at
   most 64 times it.  weights and weights_out: both or neither; they may be
   the same array, but not overlap otherwise. */
int dsv4_gqa_decode(const void* q, int64_t q_stride, int32_t type, int32_t batch, int32_t num_heads,
                    const int32_t* lens, const int32_t* req_pool_indices,
                    const dsv4_gqa_cache* cache, int32_t window, int32_t max_len,
                    const float* sink, float scale,
                    const float* weights, float* weights_out, int64_t width, float decay,
                    void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace of a decode call (0 for arguments that it refuses);
   with_weights: whether it is given weights. */
size_t dsv4_gqa_decode_workspace_size(const dsv4_gqa_cache* cache, int32_t batch, int32_t num_heads,
                                      int32_t max_len, int32_t with_weights);

/* keep >= 1, first >= 0, recent >= 0, first + recent <= keep.  seq_lens:
   tokens that each request has seen (NULL: as many as it has rows).
   positions and positions_out: both or neither.  lens_out may be lens
   or seq_lens.  Arrays that overlap otherwise are refused. */
int dsv4_gqa_evict(int32_t batch, const int32_t* lens, const int32_t* seq_lens,
                   const int32_t* req_pool_indices, const dsv4_gqa_cache* cache, int32_t max_len,
                   int32_t keep, int32_t first, int32_t recent,
                   const float* weights, float* weights_out,
                   const int32_t* positions, int32_t* positions_out, int64_t width,
                   int32_t* lens_out, void* workspace, size_t workspace_bytes, void* stream);

size_t dsv4_gqa_evict_workspace_size(const dsv4_gqa_cache* cache, int32_t batch, int32_t max_len,
                                     int32_t keep);

#ifdef __cplusplus
}
#endif

#endif /* DSV4GQA_H */
