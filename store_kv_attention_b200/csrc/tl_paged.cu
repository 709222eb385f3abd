// C ABI of the paged K/V cache (include/tl_paged.h): host-side validation and kernel launches.
#include <math.h>

#include <initializer_list>

#include "paged_internal.cuh"

namespace {

using tl::PagedBufs;
using tl::PagedShape;
using tl::set_error;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

tl_status cuda_error(cudaError_t e, const char* what) {
  return set_error(TL_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

tl_status check_desc(const tl_paged_desc* d, PagedShape* s) {
  if (!d) return set_error(TL_ERR_INVALID_ARG, "desc is NULL");
  if (d->dtype != TL_KV_FP16 && d->dtype != TL_KV_BF16)
    return set_error(TL_ERR_INVALID_ARG, "dtype %d is not a tl_kv_dtype", d->dtype);
  if (d->n_layers <= 0 || d->n_pages <= 0 || d->page_size <= 0 || d->n_kv_heads <= 0 || d->head_dim <= 0 ||
      d->max_seqs <= 0 || d->max_pages <= 0)
    return set_error(TL_ERR_INVALID_ARG, "desc has a non-positive size");
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
    return set_error(TL_ERR_UNSUPPORTED, "page_size %d not in {16, 32, 64, 128}", d->page_size);
  if (d->head_dim != 64 && d->head_dim != 128)
    return set_error(TL_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", d->head_dim);
  if (d->n_kv_heads > 256) return set_error(TL_ERR_UNSUPPORTED, "n_kv_heads %d > 256", d->n_kv_heads);
  if ((int64_t)d->max_pages * d->page_size > (1 << 22))
    return set_error(TL_ERR_UNSUPPORTED, "max_pages %d of %d positions: more than 2^22 positions", d->max_pages, d->page_size);
  if (d->n_pages > (1 << 22) || (int64_t)d->n_pages * d->n_kv_heads * d->page_size > INT32_MAX)
    return set_error(TL_ERR_UNSUPPORTED, "n_pages %d: too many pages or rows", d->n_pages);
  if (d->max_seqs > 65536) return set_error(TL_ERR_UNSUPPORTED, "max_seqs %d > 65536", d->max_seqs);
  if (d->n_layers > 65536) return set_error(TL_ERR_UNSUPPORTED, "n_layers %d > 65536", d->n_layers);
  *s = PagedShape{d->n_layers, d->n_pages,  d->page_size, d->n_kv_heads,
                  d->head_dim, d->max_seqs, d->max_pages, d->dtype};
  return TL_OK;
}

tl_status check_cache(const tl_paged_cache& c, bool need_refs) {
  if (!c.k || !c.v || !c.table) return set_error(TL_ERR_INVALID_ARG, "cache.k / v / table is NULL");
  if (need_refs && !c.refs) return set_error(TL_ERR_INVALID_ARG, "cache.refs is NULL");
  if (!aligned(c.k, 256) || !aligned(c.v, 256) || !aligned(c.table, 256) || !aligned(c.refs, 256))
    return set_error(TL_ERR_INVALID_ARG, "cache buffers must be 256-byte aligned");
  return TL_OK;
}

tl_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws) return set_error(TL_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return set_error(TL_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (bytes < need) return set_error(TL_ERR_CAPACITY, "workspace %zu bytes < %zu needed", bytes, need);
  return TL_OK;
}

tl_status check_lanes(const PagedShape& s, int32_t n_lanes, const int32_t* seqs) {
  if (n_lanes <= 0) return set_error(TL_ERR_INVALID_ARG, "n_lanes %d <= 0", n_lanes);
  if (n_lanes > tl::kPagedMaxLanes)
    return set_error(TL_ERR_UNSUPPORTED, "n_lanes %d > %d lanes per call", n_lanes, tl::kPagedMaxLanes);
  if (!seqs && n_lanes > s.max_seqs)
    return set_error(TL_ERR_CAPACITY, "n_lanes %d > max_seqs %d", n_lanes, s.max_seqs);
  return TL_OK;
}

tl_status check_heads(const PagedShape& s, int32_t n_heads) {
  if (n_heads <= 0) return set_error(TL_ERR_INVALID_ARG, "n_heads %d <= 0", n_heads);
  if (n_heads % s.kv != 0)
    return set_error(TL_ERR_SHAPE, "n_heads %d is not a multiple of n_kv_heads %d", n_heads, s.kv);
  if (n_heads > 1024) return set_error(TL_ERR_UNSUPPORTED, "n_heads %d > 1024", n_heads);
  return TL_OK;
}

tl_status check_split(int32_t split_rows) {
  if (split_rows < 0 || split_rows > 4096 || split_rows % 128 != 0)
    return set_error(TL_ERR_INVALID_ARG, "split_rows %d is not 0 or a multiple of 128 up to 4096", split_rows);
  return TL_OK;
}

// Row stride in elements: 0 = dense.
tl_status check_stride(int64_t* stride, int64_t dense, const char* what) {
  if (*stride == 0) *stride = dense;
  if (*stride < dense || *stride % 8 != 0 || *stride >= ((int64_t)1 << 38))
    return set_error(TL_ERR_INVALID_ARG, "%s %lld is not a multiple of 8 that is at least %lld", what,
                     (long long)*stride, (long long)dense);
  return TL_OK;
}

tl_status check_layer(const PagedShape& s, int32_t layer) {
  if (layer < 0 || layer >= s.layers) return set_error(TL_ERR_CAPACITY, "layer %d outside [0, %d)", layer, s.layers);
  return TL_OK;
}

tl_status check_scale(float* scale, int hd) {
  if (!(*scale >= 0.0f) || isinf(*scale)) return set_error(TL_ERR_INVALID_ARG, "scale must be finite and not negative");
  if (*scale == 0.0f) *scale = 1.0f / sqrtf((float)hd);
  return TL_OK;
}

PagedBufs bufs(const tl_paged_cache& c) { return PagedBufs{(uint16_t*)c.k, (uint16_t*)c.v, c.table, c.refs}; }

// What the operations on pages have in common.
tl_status check_op(const tl_paged_desc* desc, const tl_paged_cache& c, int32_t n, int32_t most, const void* ws,
                   size_t bytes, PagedShape* s) {
  tl_status st = check_desc(desc, s);
  if (st != TL_OK) return st;
  if ((st = check_cache(c, true)) != TL_OK) return st;
  if (n < 0) return set_error(TL_ERR_INVALID_ARG, "n %d < 0", n);
  if (n > most) return set_error(TL_ERR_UNSUPPORTED, "n %d > %d in one call", n, most);
  return check_workspace(ws, bytes, tl::paged_ops_workspace(*s).total);
}

}  // namespace

extern "C" {

tl_status tl_paged_cache_bytes(const tl_paged_desc* desc, size_t* pool_bytes, size_t* table_bytes,
                               size_t* refs_bytes) {
  PagedShape s{};
  tl_status st = check_desc(desc, &s);
  if (st != TL_OK) return st;
  if (!pool_bytes || !table_bytes || !refs_bytes) return set_error(TL_ERR_INVALID_ARG, "output pointer is NULL");
  *pool_bytes = (size_t)s.layers * s.layer_elems() * 2;
  *table_bytes = (size_t)s.max_seqs * s.max_pages * 4;
  *refs_bytes = (size_t)s.n_pages * 4;
  return TL_OK;
}

tl_status tl_paged_workspace_bytes(const tl_paged_desc* desc, int32_t n_heads, int32_t n_lanes, int32_t split_rows,
                                   size_t* bytes) {
  PagedShape s{};
  tl_status st = check_desc(desc, &s);
  if (st != TL_OK) return st;
  if (!bytes) return set_error(TL_ERR_INVALID_ARG, "bytes is NULL");
  if ((st = check_heads(s, n_heads)) != TL_OK) return st;
  if (n_lanes <= 0) return set_error(TL_ERR_INVALID_ARG, "n_lanes %d <= 0", n_lanes);
  if (n_lanes > tl::kPagedMaxLanes)
    return set_error(TL_ERR_UNSUPPORTED, "n_lanes %d > %d lanes per call", n_lanes, tl::kPagedMaxLanes);
  if ((st = check_split(split_rows)) != TL_OK) return st;
  size_t most = tl::paged_workspace_upto(s, n_heads, n_lanes, split_rows);
  for (const size_t need : {tl::paged_ops_workspace(s).total, tl::prompt_plan(s, n_heads, 1, 1).total})
    if (need > most) most = need;
  *bytes = most;
  return TL_OK;
}

tl_status tl_paged_append(const tl_paged_desc* desc, tl_paged_cache cache, int32_t layer, const void* k_rows,
                          int64_t k_stride, const void* v_rows, int64_t v_stride, int32_t n_rows,
                          const int32_t* cu_rows, const int32_t* start_pos, const int32_t* seqs, int32_t n_lanes,
                          void* workspace, size_t workspace_bytes, tl_stream_t stream) {
  PagedShape s{};
  tl_status st = check_desc(desc, &s);
  if (st != TL_OK) return st;
  if ((st = check_cache(cache, false)) != TL_OK) return st;
  if (n_rows < 0) return set_error(TL_ERR_INVALID_ARG, "n_rows %d < 0", n_rows);
  if (n_rows == 0) return check_layer(s, layer);  // nothing to write (an empty array may have no address)
  if (!k_rows || !v_rows || !start_pos) return set_error(TL_ERR_INVALID_ARG, "k_rows / v_rows / start_pos is NULL");
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16))
    return set_error(TL_ERR_INVALID_ARG, "k_rows and v_rows must be 16-byte aligned");
  if ((st = check_layer(s, layer)) != TL_OK) return st;
  if ((st = check_lanes(s, n_lanes, seqs)) != TL_OK) return st;
  if (!cu_rows && n_rows != n_lanes)
    return set_error(TL_ERR_INVALID_ARG, "n_rows %d != n_lanes %d without cu_rows", n_rows, n_lanes);
  const int64_t dense = (int64_t)s.kv * s.hd;
  if ((st = check_stride(&k_stride, dense, "k_stride")) != TL_OK) return st;
  if ((st = check_stride(&v_stride, dense, "v_stride")) != TL_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, 256)) != TL_OK) return st;
  cudaError_t e = tl::launch_paged_append(s, bufs(cache), layer, k_rows, k_stride, v_rows, v_stride, n_rows, cu_rows,
                                          start_pos, seqs, n_lanes, (uint32_t*)workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "tl_paged_append launch");
  return TL_OK;
}

tl_status tl_paged_attn_decode(const tl_paged_desc* desc, tl_paged_cache cache, int32_t layer, int32_t n_heads,
                               const void* q, int64_t q_stride, const int32_t* kv_len, const int32_t* seqs,
                               float scale, int32_t split_rows, void* out, int32_t n_lanes, void* workspace,
                               size_t workspace_bytes, tl_stream_t stream) {
  PagedShape s{};
  tl_status st = check_desc(desc, &s);
  if (st != TL_OK) return st;
  if ((st = check_cache(cache, false)) != TL_OK) return st;
  if (!q || !kv_len || !out) return set_error(TL_ERR_INVALID_ARG, "q / kv_len / out is NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return set_error(TL_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if ((st = check_layer(s, layer)) != TL_OK) return st;
  if ((st = check_heads(s, n_heads)) != TL_OK) return st;
  if ((st = check_lanes(s, n_lanes, seqs)) != TL_OK) return st;
  if ((st = check_stride(&q_stride, (int64_t)n_heads * s.hd, "q_stride")) != TL_OK) return st;
  if ((st = check_scale(&scale, s.hd)) != TL_OK) return st;
  if ((st = check_split(split_rows)) != TL_OK) return st;
  const tl::PagedWorkspace wl = tl::paged_workspace(s, n_heads, n_lanes, split_rows);
  if ((st = check_workspace(workspace, workspace_bytes, wl.total)) != TL_OK) return st;
  if ((int64_t)n_lanes * wl.s_max * tl::paged_tiles(s, n_heads) > INT32_MAX)
    return set_error(TL_ERR_UNSUPPORTED, "%d lanes of %d splits in one call", n_lanes, wl.s_max);
  const tl::PagedDecodeArgs a{s, bufs(cache), layer, n_heads, n_lanes, q, q_stride, kv_len,
                              seqs, scale, out, (uint8_t*)workspace, wl};
  cudaError_t e = tl::launch_paged_decode(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "tl_paged_attn_decode launch");
  return TL_OK;
}

tl_status tl_paged_prompt_attn(const tl_paged_desc* desc, tl_paged_cache cache, int32_t layer, int32_t n_heads,
                               const void* q, int64_t q_stride, int32_t n_rows, const int32_t* cu_q,
                               const int32_t* kv_len, const int32_t* seqs, float scale, void* out, int32_t n_lanes,
                               void* workspace, size_t workspace_bytes, tl_stream_t stream) {
  PagedShape s{};
  tl_status st = check_desc(desc, &s);
  if (st != TL_OK) return st;
  if ((st = check_cache(cache, false)) != TL_OK) return st;
  if (n_rows < 0) return set_error(TL_ERR_INVALID_ARG, "n_rows %d < 0", n_rows);
  if (n_rows == 0) return check_layer(s, layer);  // no queries
  if (!q || !cu_q || !kv_len || !out) return set_error(TL_ERR_INVALID_ARG, "q / cu_q / kv_len / out is NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return set_error(TL_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if ((st = check_layer(s, layer)) != TL_OK) return st;
  if ((st = check_heads(s, n_heads)) != TL_OK) return st;
  if ((st = check_lanes(s, n_lanes, seqs)) != TL_OK) return st;
  if (n_rows > (1 << 24)) return set_error(TL_ERR_UNSUPPORTED, "n_rows %d > 2^24", n_rows);
  if ((st = check_stride(&q_stride, (int64_t)n_heads * s.hd, "q_stride")) != TL_OK) return st;
  if ((st = check_scale(&scale, s.hd)) != TL_OK) return st;
  const tl::PromptPlan plan = tl::prompt_plan(s, n_heads, n_lanes, n_rows);
  if ((st = check_workspace(workspace, workspace_bytes, plan.total)) != TL_OK) return st;
  if (plan.blocks > INT32_MAX / 16)
    return set_error(TL_ERR_UNSUPPORTED, "%d rows of %d heads in one call", n_rows, n_heads);
  const tl::PagedPromptArgs a{s, bufs(cache), layer, n_heads, n_lanes, n_rows, q, q_stride, cu_q,
                              kv_len, seqs, scale, out, (uint8_t*)workspace, plan};
  cudaError_t e = tl::launch_paged_prompt(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "tl_paged_prompt_attn launch");
  return TL_OK;
}

tl_status tl_paged_copy(const tl_paged_desc* desc, tl_paged_cache cache, const int32_t* src, const int32_t* dst,
                        int32_t n, void* workspace, size_t workspace_bytes, tl_stream_t stream) {
  PagedShape s{};
  tl_status st = check_op(desc, cache, n, desc ? desc->n_pages : 0, workspace, workspace_bytes, &s);
  if (st != TL_OK) return st;
  if (n == 0) return TL_OK;
  if (!src || !dst) return set_error(TL_ERR_INVALID_ARG, "src / dst is NULL");
  cudaError_t e = tl::launch_paged_copy(s, bufs(cache), src, dst, n, (uint8_t*)workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "tl_paged_copy launch");
  return TL_OK;
}

tl_status tl_paged_fork(const tl_paged_desc* desc, tl_paged_cache cache, const int32_t* src, const int32_t* dst,
                        const int32_t* n_tokens, int32_t n, void* workspace, size_t workspace_bytes,
                        tl_stream_t stream) {
  PagedShape s{};
  tl_status st = check_op(desc, cache, n, tl::kPagedMaxLanes, workspace, workspace_bytes, &s);
  if (st != TL_OK) return st;
  if (n == 0) return TL_OK;
  if (!src || !dst || !n_tokens) return set_error(TL_ERR_INVALID_ARG, "src / dst / n_tokens is NULL");
  cudaError_t e = tl::launch_paged_fork(s, bufs(cache), src, dst, n_tokens, n, (uint8_t*)workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "tl_paged_fork launch");
  return TL_OK;
}

tl_status tl_paged_reserve(const tl_paged_desc* desc, tl_paged_cache cache, const int32_t* seqs,
                           const int32_t* ctx_len, const int32_t* n_new, int32_t n, void* workspace,
                           size_t workspace_bytes, tl_stream_t stream) {
  PagedShape s{};
  tl_status st = check_op(desc, cache, n, tl::kPagedMaxLanes, workspace, workspace_bytes, &s);
  if (st != TL_OK) return st;
  if (n == 0) return TL_OK;
  if (!seqs || !ctx_len || !n_new) return set_error(TL_ERR_INVALID_ARG, "seqs / ctx_len / n_new is NULL");
  cudaError_t e = tl::launch_paged_reserve(s, bufs(cache), seqs, ctx_len, n_new, n, (uint8_t*)workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "tl_paged_reserve launch");
  return TL_OK;
}

tl_status tl_paged_free(const tl_paged_desc* desc, tl_paged_cache cache, const int32_t* seqs, const int32_t* keep,
                        int32_t n, void* workspace, size_t workspace_bytes, tl_stream_t stream) {
  PagedShape s{};
  tl_status st = check_op(desc, cache, n, tl::kPagedMaxLanes, workspace, workspace_bytes, &s);
  if (st != TL_OK) return st;
  if (n == 0) return TL_OK;
  if (!seqs) return set_error(TL_ERR_INVALID_ARG, "seqs is NULL");
  cudaError_t e = tl::launch_paged_free(s, bufs(cache), seqs, keep, n, (uint8_t*)workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "tl_paged_free launch");
  return TL_OK;
}

tl_status tl_paged_compact(const tl_paged_desc* desc, tl_paged_cache cache, int32_t* n_live, void* workspace,
                           size_t workspace_bytes, tl_stream_t stream) {
  PagedShape s{};
  tl_status st = check_op(desc, cache, 0, 0, workspace, workspace_bytes, &s);
  if (st != TL_OK) return st;
  cudaError_t e = tl::launch_paged_compact(s, bufs(cache), n_live, (uint8_t*)workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "tl_paged_compact launch");
  return TL_OK;
}

}  // extern "C"
