// Rows of K and V into the paged cache (tl_paged_append).
//
// A copy: row r of the packed input, [kv][hd] of K and of V, goes to the page of its position, one
// run of hd values per K/V head.  Bytes (2 x 2 x n_rows x kv x hd x 2) bound it; a call of single
// tokens is bound by its chain of dependent loads (cu_rows, start_pos, table, refs, then the rows).
// One warp takes 2 KB of K or of V of one row, so that a lane has four 16-byte loads in flight and a
// 48-token call still spreads over as many warps as it has parts.  Measured: 24 packed prompts of up to 2048
// rows of 8 x 128, 204 MB in 34.5 us a call, 5.9 TB/s (0.91 of a copy's bandwidth; at 32 registers, twice the warps,
// 37.3); 48 tokens 6.5 us a call, most of it the host's.
#include "paged_internal.cuh"
#include "tc_ptx.cuh"

namespace tl {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kPart = 128;  // 16-byte chunks of one row a warp takes at a time

// The lane that owns packed row r: the largest b with cu[b] <= r, for cu[0] <= r < cu[n].  All lanes
// of the warp search together, 32 bounds a step.  Any contents of cu give a b in [0, n).
__device__ __forceinline__ int find_lane(const int32_t* cu, int n, int r, int lane) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && (lane == 0 || cu[at] <= r));
    lo += (31 - __clz(le)) * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  return lo;
}

__global__ void __launch_bounds__(kAppendThreads)
    paged_append_kernel(PagedShape s, PagedBufs c, size_t layer_off, const uint16_t* k_rows, int64_t k_stride,
                        const uint16_t* v_rows, int64_t v_stride, int n_rows, const int32_t* cu_rows,
                        const int32_t* start_pos, const int32_t* seqs, int n_lanes, uint32_t* status) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int lane = threadIdx.x & 31, part = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int chunks = s.kv * s.hd / 8, log_page = 31 - __clz(s.page), log_head = s.hd == 64 ? 3 : 4;  // 16-byte chunks
  int first = 0, last = n_rows;
  if (cu_rows) {
    first = max(0, cu_rows[0]);
    last = min(n_rows, cu_rows[n_lanes]);
  }
  const int step = gridDim.x * (kAppendThreads / 32);
  for (long long at_row = (long long)first + blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5); at_row < last; at_row += step) {
    const int r = (int)at_row;
    // the row's values are on their way while its place is looked up
    const uint4* src = reinterpret_cast<const uint4*>(is_v ? v_rows + r * v_stride : k_rows + r * k_stride);
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = part * kPart + i * 32 + lane;
      if (at < chunks) x[i] = __ldg(src + at);
    }
    const int b = cu_rows ? find_lane(cu_rows, n_lanes, r, lane) : r;
    const int seq = seqs ? seqs[b] : b;
    const int own0 = cu_rows ? cu_rows[b] : r, own1 = cu_rows ? cu_rows[b + 1] : r + 1;  // the lane's rows
    const long long pos = (long long)start_pos[b] + r - own0;
    bool ok = seq >= 0 && seq < s.max_seqs && pos >= 0 && pos < s.max_len();
    ok = ok && own0 >= 0 && own0 <= r && r < own1 && own1 <= n_rows;
    int page = -1;
    if (ok) page = c.table[(size_t)seq * s.max_pages + (int)(pos >> log_page)];
    ok = ok && page >= 0 && page < s.n_pages;
    if (ok && c.refs) ok = c.refs[page] <= 1;
    if (!ok) {
      if (lane == 0) atomicOr(status, kStatusRange);
      continue;
    }
    uint16_t* dst = (is_v ? c.v : c.k) + layer_off + (size_t)page * s.page_elems() + (size_t)((int)pos & (s.page - 1)) * s.hd;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = part * kPart + i * 32 + lane;
      if (at < chunks) *reinterpret_cast<uint4*>(dst + (size_t)(at >> log_head) * s.block_elems() + (at & ((1 << log_head) - 1)) * 8) = x[i];
    }
  }
  // a lane may claim rows that no warp above has met: one block looks the lanes over
  if (cu_rows && blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < n_lanes; b += kAppendThreads)
      if (cu_rows[b] < 0 || cu_rows[b + 1] < cu_rows[b] || cu_rows[b + 1] > n_rows) atomicOr(status, kStatusRange);
}

}  // namespace

cudaError_t launch_paged_append(const PagedShape& s, const PagedBufs& c, int layer, const void* k_rows, int64_t k_stride,
                                const void* v_rows, int64_t v_stride, int n_rows, const int32_t* cu_rows,
                                const int32_t* start_pos, const int32_t* seqs, int n_lanes, uint32_t* status,
                                cudaStream_t st) {
  const int parts = (s.kv * s.hd / 8 + kPart - 1) / kPart;
  const long long blocks = ((long long)n_rows + kAppendThreads / 32 - 1) / (kAppendThreads / 32), most = (148 * 8 + 2 * parts - 1) / (2 * parts);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most), 2 * parts);
  cfg.blockDim = dim3(kAppendThreads);
  cudaError_t e = cudaLaunchKernelEx(&cfg, paged_append_kernel, s, c, (size_t)layer * s.layer_elems(),
                                     (const uint16_t*)k_rows, k_stride, (const uint16_t*)v_rows, v_stride, n_rows,
                                     cu_rows, start_pos, seqs, n_lanes, status);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tl
