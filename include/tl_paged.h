/*
 * tl_paged.h -- paged cache of K and V: layout, append, single-token and prompt attention, and
 * the operations on its pages.
 *
 * The store-h cache (tl_storeh.h) serves the loop block, whose iterations share one W_k and W_v.
 * The n_pre unique layers before it have weights of their own and attend stored K and V; the
 * pages name paged attention and chunked prefill for them [Architecture-Exclusive Features,
 * "What this list is not"].  This header is that cache: fixed-size pages of positions in one
 * pool, a page table per sequence, and a count of the sequences that hold each page, so that
 * sequences of different lengths share memory and forked sequences share their common prefix.
 *
 * Attention, per lane b and query head h (K/V head g = h / (n_heads / n_kv_heads)):
 *     out = sum_c softmax_c(scale * q . k_c) v_c      over the positions c the query attends
 * with the statistics and the sum in FP32; a query that attends nothing gives zeros.  The softmax
 * weights enter the second product rounded to the cache's 16-bit type, like the output: half a step,
 * and in FP16 at least 2^-32 of the largest weight.
 *
 * Conventions are those of tl_storeh.h: caller-owned device memory on the current device,
 * asynchronous on a stream, host-side validation before any launch (a non-TL_OK return enqueues
 * nothing, except TL_ERR_CUDA for a failed launch), programmatic dependent launch with stream
 * order preserved, tl_last_error_message() for details.  Values read from device arrays are
 * checked on the device: what is out of range is skipped as each call says and
 * TL_ERR_DEVICE_RANGE is recorded in the workspace's status word (tl_storeh_poll_status).
 *
 * Every call takes the workspace of tl_paged_workspace_bytes (256-byte aligned, its first 4096
 * bytes zeroed once; the status word is its first).  Calls on one stream may share a workspace,
 * and so may captured graphs that are replayed one after the other; calls that may overlap on
 * the GPU need one each, except tl_paged_append, tl_paged_fork and tl_paged_free, which touch
 * only the status word.  After TL_ERR_DEVICE_TIMEOUT the 4096 bytes are to be zeroed again.
 */
#ifndef TL_PAGED_H_
#define TL_PAGED_H_

#include "tl_storeh.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a paged cache, of the queries that attend it and of their outputs. */
typedef enum {
  TL_KV_FP16 = 0,
  TL_KV_BF16 = 1
} tl_kv_dtype;

/* Shape of one paged cache.  Supported: page_size in {16, 32, 64, 128}; head_dim in {64, 128};
 * n_kv_heads <= 256; max_pages * page_size <= 2^22 positions per sequence; n_pages <= 2^22 and
 * n_pages * n_kv_heads * page_size <= 2^31 - 1; max_seqs <= 65536. */
typedef struct {
  int32_t n_layers;   /* page p of every layer belongs to the same positions of the same sequences */
  int32_t n_pages;    /* pages in the pool */
  int32_t page_size;  /* positions per page */
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t max_seqs;   /* rows of the page table */
  int32_t max_pages;  /* page-table entries per sequence */
  int32_t dtype;      /* tl_kv_dtype */
} tl_paged_desc;

/* Device buffers, caller-allocated, each 256-byte aligned:
 *   k, v   [n_layers][n_pages][n_kv_heads][page_size][head_dim]  fp16 or bf16
 *   table  int32 [max_seqs][max_pages]: entry j of row s is the page of positions
 *          j * page_size .. of sequence s, -1 = none; -1 everywhere to begin with
 *   refs   int32 [n_pages]: table entries that name the page, 0 = free; 0 everywhere to begin
 *          with.  NULL for a caller that keeps its page table itself: append, decode and prompt
 *          attention then take the table as it is, the operations on pages are refused. */
typedef struct {
  void* k;
  void* v;
  int32_t* table;
  int32_t* refs;
} tl_paged_cache;

/* Sizes in bytes of k (and of v), table and refs.
 * Errors: TL_ERR_INVALID_ARG (NULL, non-positive size, dtype), TL_ERR_UNSUPPORTED. */
TL_API tl_status tl_paged_cache_bytes(const tl_paged_desc* desc, size_t* pool_bytes, size_t* table_bytes,
                                      size_t* refs_bytes);

/* Workspace bytes for calls of up to n_lanes lanes (sequences) of n_heads query heads and split
 * length split_rows (see tl_paged_attn_decode), for prompt attention over any number of rows
 * (59 MB at head_dim 128: partial results of 444 pieces) and for the operations on pages.
 * Errors: the desc errors, TL_ERR_INVALID_ARG (n_lanes, n_heads not positive, split_rows),
 * TL_ERR_SHAPE (n_heads not a multiple of n_kv_heads), TL_ERR_UNSUPPORTED (n_lanes > 1024,
 * n_heads > 1024). */
TL_API tl_status tl_paged_workspace_bytes(const tl_paged_desc* desc, int32_t n_heads, int32_t n_lanes,
                                          int32_t split_rows, size_t* bytes);

/*
 * Writes rows of K and V into layer `layer`.
 *   k_rows, v_rows  device [n_rows][n_kv_heads][head_dim], row r at r * k_stride (v_stride)
 *                   elements: a multiple of 8 and at least n_kv_heads * head_dim, or 0 for that
 *                   (so parts of one projection's output can be passed as they are); 16-byte aligned
 *   cu_rows   device int32 [n_lanes + 1], not decreasing, or NULL: lane b owns rows
 *             cu_rows[b] .. cu_rows[b+1] - 1 (packed prompts); NULL: one row per lane
 *             (n_rows = n_lanes).  Rows outside [cu_rows[0], cu_rows[n_lanes]) are not used.
 *   start_pos device int32 [n_lanes]: lane b's row i goes to position start_pos[b] + i
 *   seqs      device int32 [n_lanes] or NULL: the sequence (table row) of each lane; NULL: lane b
 *             is sequence b
 * No two rows of a call may go to the same position.
 * A row whose sequence or position is out of range, whose page is not in the table, or whose page
 * is held by more than one sequence (refs > 1: tl_paged_reserve gives the writer its own) is not
 * written, nor are the rows of a lane that begins before row 0, ends before it begins or ends past
 * n_rows; TL_ERR_DEVICE_RANGE is recorded.
 * Errors: TL_ERR_INVALID_ARG, TL_ERR_CAPACITY (layer, n_lanes > max_seqs without seqs, workspace),
 * TL_ERR_UNSUPPORTED, TL_ERR_CUDA.
 */
TL_API tl_status tl_paged_append(const tl_paged_desc* desc, tl_paged_cache cache, int32_t layer, const void* k_rows,
                                 int64_t k_stride, const void* v_rows, int64_t v_stride, int32_t n_rows,
                                 const int32_t* cu_rows, const int32_t* start_pos, const int32_t* seqs,
                                 int32_t n_lanes, void* workspace, size_t workspace_bytes, tl_stream_t stream);

/*
 * One new token per lane: query q[b] attends positions 0 .. kv_len[b] - 1 of its sequence in
 * layer `layer` (its own position among them, appended before).
 *   q        device [n_lanes][n_heads][head_dim], lane b at b * q_stride elements (a multiple of
 *            8, at least n_heads * head_dim, or 0 for that), 16-byte aligned
 *   kv_len   device int32 [n_lanes]; 0 gives zeros
 *   out      device [n_lanes][n_heads][head_dim] in the cache's type, 16-byte aligned
 *   scale    the softmax scale, > 0 and finite, or 0 for 1 / sqrt(head_dim)
 *   split_rows  positions per split, 0 or a multiple of 128 up to 4096.  A lane's positions are
 *            cut into splits that run side by side and are joined exactly.  0 takes a length by
 *            the lane's own kv_len and by how many (lane, K/V head) pairs the call has for the
 *            GPU's SMs; a lane's result then depends, by the order of its sums, on n_lanes.  With
 *            a length given, it depends on its own rows alone, as in tl_storeh_decode_ex.
 * A lane whose sequence or kv_len is out of range ([0, max_pages * page_size]) is skipped (its
 * out rows are not written); positions whose table entry names no page of the pool are left out.
 * Both record TL_ERR_DEVICE_RANGE.
 * Errors: TL_ERR_INVALID_ARG, TL_ERR_SHAPE (n_heads not a multiple of n_kv_heads),
 * TL_ERR_CAPACITY (layer, n_lanes > max_seqs without seqs, workspace too small),
 * TL_ERR_UNSUPPORTED, TL_ERR_CUDA.
 */
TL_API tl_status tl_paged_attn_decode(const tl_paged_desc* desc, tl_paged_cache cache, int32_t layer, int32_t n_heads,
                                      const void* q, int64_t q_stride, const int32_t* kv_len, const int32_t* seqs,
                                      float scale, int32_t split_rows, void* out, int32_t n_lanes, void* workspace,
                                      size_t workspace_bytes, tl_stream_t stream);

/*
 * Prompts, packed: lane b's queries are rows cu_q[b] .. cu_q[b+1] - 1 of q, the newest of its
 * kv_len[b] positions; query i (of n = cu_q[b+1] - cu_q[b]) sits at position kv_len[b] - n + i and
 * attends positions 0 .. itself.  A whole prompt has kv_len[b] = n; a chunk of one, or a prompt
 * behind a shared prefix, more.  K and V were appended before (tl_paged_append).
 *   q      device [n_rows][n_heads][head_dim], row r at r * q_stride elements as above
 *   cu_q   device int32 [n_lanes + 1], not decreasing, 0 <= cu_q[0], cu_q[n_lanes] <= n_rows
 *   out    device [n_rows][n_heads][head_dim]; rows outside every lane are not written
 * Queries at negative positions (kv_len[b] < n) attend nothing and give zeros.  Values of K and V
 * at positions a query does not attend never reach its output, whatever they are.
 * A lane whose sequence, kv_len or rows are out of range, or any of whose kv_len positions has no
 * page of the pool, is skipped (its out rows are not written) and TL_ERR_DEVICE_RANGE recorded.
 * Errors: as tl_paged_attn_decode.
 */
TL_API tl_status tl_paged_prompt_attn(const tl_paged_desc* desc, tl_paged_cache cache, int32_t layer, int32_t n_heads,
                                      const void* q, int64_t q_stride, int32_t n_rows, const int32_t* cu_q,
                                      const int32_t* kv_len, const int32_t* seqs, float scale, void* out,
                                      int32_t n_lanes, void* workspace, size_t workspace_bytes, tl_stream_t stream);

/*
 * Operations on pages.  Each acts on every layer's K and V.  Results do not depend on scheduling:
 * pages are taken lowest index first, in the order of the lists.
 * Errors of all: TL_ERR_INVALID_ARG (refs NULL too), TL_ERR_CAPACITY (workspace),
 * TL_ERR_UNSUPPORTED (more than 1024 sequences in one call), TL_ERR_CUDA.
 */

/* Copies page src[i] to page dst[i], i < n (device int32 [n]; n <= n_pages).  The table and refs
 * stay as they are.  Pair i is skipped, and TL_ERR_DEVICE_RANGE recorded, when a page is out of
 * range, when dst[i] is the destination of an earlier pair, or when src[i] is any pair's
 * destination. */
TL_API tl_status tl_paged_copy(const tl_paged_desc* desc, tl_paged_cache cache, const int32_t* src, const int32_t* dst,
                               int32_t n, void* workspace, size_t workspace_bytes, tl_stream_t stream);

/* Makes sequence dst[i] share the first n_tokens[i] positions of sequence src[i] (device int32
 * [n] each): their pages, the partly filled last one among them, are entered in dst[i]'s row and
 * counted.  Nothing is copied; tl_paged_reserve copies a shared page before it is written.
 * Fork i is skipped, and TL_ERR_DEVICE_RANGE recorded, when a sequence or length is out of range,
 * when src[i] lacks one of the pages, when dst[i] holds a page, when dst[i] stands in the list
 * before, or when src[i] is any fork's dst. */
TL_API tl_status tl_paged_fork(const tl_paged_desc* desc, tl_paged_cache cache, const int32_t* src, const int32_t* dst,
                               const int32_t* n_tokens, int32_t n, void* workspace, size_t workspace_bytes,
                               tl_stream_t stream);

/* Makes positions ctx_len[i] .. ctx_len[i] + n_new[i] - 1 of sequence seqs[i] writable (device
 * int32 [n] each): an entry there without a page gets a free one; a page held by more than one
 * sequence is replaced by a free page, with a copy of its rows where the page begins before
 * ctx_len[i].  Every listed sequence that shares such a page gets its own.  Sequences are served
 * in the order of the list while the free pages last; the first one that they do not cover and
 * all behind it get nothing, and TL_ERR_DEVICE_CAPACITY is recorded (tl_storeh_poll_status returns
 * it before a TL_ERR_DEVICE_RANGE, such as that of an append to the missing pages).  A sequence that
 * is out of range, stands in the list before, has a negative length, or whose positions do not fit
 * its table row gets nothing, and TL_ERR_DEVICE_RANGE is recorded. */
TL_API tl_status tl_paged_reserve(const tl_paged_desc* desc, tl_paged_cache cache, const int32_t* seqs,
                                  const int32_t* ctx_len, const int32_t* n_new, int32_t n, void* workspace,
                                  size_t workspace_bytes, tl_stream_t stream);

/* Takes the pages behind the first keep[i] positions (NULL: all pages) out of the row of sequence
 * seqs[i] (device int32 [n] each); a page that no sequence holds any more is free.  A sequence out
 * of range or a negative keep is skipped and TL_ERR_DEVICE_RANGE recorded. */
TL_API tl_status tl_paged_free(const tl_paged_desc* desc, tl_paged_cache cache, const int32_t* seqs,
                               const int32_t* keep, int32_t n, void* workspace, size_t workspace_bytes,
                               tl_stream_t stream);

/* Moves pages so that the n pages in use are pages 0 .. n - 1: the k-th lowest page in use at or
 * above n takes the place of the k-th lowest free page below n; table and refs follow, and
 * n_live (device int32 [1], or NULL) receives n.  The rows of freed pages keep their contents. */
TL_API tl_status tl_paged_compact(const tl_paged_desc* desc, tl_paged_cache cache, int32_t* n_live, void* workspace,
                                  size_t workspace_bytes, tl_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TL_PAGED_H_ */
