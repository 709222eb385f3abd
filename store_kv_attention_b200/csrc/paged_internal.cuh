// Internal declarations of the paged K/V cache (include/tl_paged.h): shape, workspace layout and
// launchers.
#pragma once

#include "tl_internal.cuh"
#include "tl_paged.h"

namespace tl {

constexpr int kPagedMaxLanes = 1024;  // lanes (sequences) per call: the plans keep one word per lane in shared memory

struct PagedShape {
  int layers, n_pages, page, kv, hd, max_seqs, max_pages, dtype;
  __host__ __device__ size_t block_elems() const { return (size_t)page * hd; }           // one (page, K/V head)
  __host__ __device__ size_t page_elems() const { return (size_t)kv * page * hd; }       // one page of a layer
  __host__ __device__ size_t layer_elems() const { return (size_t)n_pages * page_elems(); }
  __host__ __device__ int max_len() const { return max_pages * page; }
};

// The cache's buffers as the kernels take them.
struct PagedBufs {
  uint16_t* k;
  uint16_t* v;
  int32_t* table;
  int32_t* refs;
};

// Splits of one lane's `len` positions.  target 0: splits of `rows` positions.  Otherwise target = the splits a
// lane should have so that the call fills the GPU, `rows` = the most positions of a split: as many splits as the
// two ask for, at most one per kSplitLeast positions, of equal length rounded up to 16 positions (a warp's unit).
constexpr int kSplitLeast = 128;
__host__ __device__ inline int paged_split_rows(int len, int target, int rows) {
  if (target == 0) return rows;
  const int fine = (len + kSplitLeast - 1) / kSplitLeast, coarse = (len + rows - 1) / rows;
  int n = fine < target ? fine : target;
  n = n > coarse ? n : coarse;
  n = n > 1 ? n : 1;
  const int each = (len + n - 1) / n;
  return each <= 16 ? 16 : (each + 15) / 16 * 16;
}
__host__ __device__ inline int paged_splits(int len, int target, int rows) {
  const int each = paged_split_rows(len, target, rows);
  return len <= each ? 1 : (len + each - 1) / each;
}
// The most positions of a split: 1024 (32 lanes of 4097: 178 us a call, 186 at 2048, 192 at 512; 48 lanes of up to
// 8192: 142, 148, 151), or more where a call's lanes, were they all as long as the table allows, would have more
// than 2^18 partial results.
constexpr int kSplitMost = 1024, kMostParts = 1 << 18;
inline int paged_split_most(int max_len, int n_heads, int n_lanes) {
  const long long parts = (long long)n_lanes * n_heads * ((max_len + kSplitMost - 1) / kSplitMost);
  return kSplitMost * (int)((parts + kMostParts - 1) / kMostParts);
}

// Workspace: a head that is zero between calls (status word | work queue of the prompt attention |
// finished pieces of its blocks), then, one over the other: per-split (max, sum) and unnormalised sums
// of the decode; partial results of the prompt attention; the plan of the operations on pages (counters |
// moves: source, destination | one word per page).
constexpr int kPagedQueueOff = 128, kPagedHead = 4096;
struct PagedWorkspace {
  size_t ml_off, acc_off, total;  // decode
  int s_max, target, rows;        // splits a lane can have; paged_split_rows' arguments
};
// K/V heads times tiles of 16 query heads: the CTAs that one split of one lane takes.
inline int paged_tiles(const PagedShape& s, int n_heads) { return s.kv * ((n_heads / s.kv + 15) / 16); }
constexpr int kPagedSlots = 296;  // two CTAs on each of the 148 SMs
inline PagedWorkspace paged_workspace(const PagedShape& s, int n_heads, int n_lanes, int split_rows) {
  PagedWorkspace w;
  const int pairs = n_lanes * paged_tiles(s, n_heads), len = s.max_len();
  w.target = split_rows ? 0 : (kPagedSlots + pairs - 1) / pairs;
  w.rows = split_rows ? split_rows : paged_split_most(len, n_heads, n_lanes);
  const int fine = (len + kSplitLeast - 1) / kSplitLeast, coarse = (len + w.rows - 1) / w.rows;
  w.s_max = w.target < fine ? w.target : fine;
  if (w.s_max < coarse) w.s_max = coarse;
  const size_t parts = (size_t)n_lanes * n_heads * w.s_max;
  w.ml_off = kPagedHead;
  w.acc_off = align256(w.ml_off + parts * 8);
  w.total = align256(w.acc_off + parts * s.hd * 4);
  return w;
}
// Enough for every call of up to n_lanes lanes.  With fewer lanes a lane has more splits, but
// n * ceil(slots / (n * tiles)) never passes slots / tiles + n, nor n * heads * ceil(len / most) the larger of
// kMostParts + n * heads and the parts of 1024 positions.
inline size_t paged_workspace_upto(const PagedShape& s, int n_heads, int n_lanes, int split_rows) {
  const size_t len = s.max_len(), lanes = n_lanes;
  const size_t fine = lanes * ((len + kSplitLeast - 1) / kSplitLeast) * n_heads;
  size_t coarse = lanes * ((len + kSplitMost - 1) / kSplitMost) * n_heads;
  if (coarse > kMostParts + lanes * n_heads) coarse = kMostParts + lanes * n_heads;
  size_t parts = (kPagedSlots / paged_tiles(s, n_heads) + 1 + lanes) * n_heads;
  if (parts > fine) parts = fine;
  if (parts < coarse) parts = coarse;
  if (split_rows) parts = lanes * ((len + split_rows - 1) / split_rows) * n_heads;
  return align256(align256(kPagedHead + parts * 8) + parts * s.hd * 4);
}
// Prompt attention: heads packed into a tile's rows (the largest power of two up to 128 that divides the
// group), blocks of two tiles there can be, and the most pieces that a block may be cut into (a piece has at
// least kPieceSteps steps of 64 positions; a call has at most kPromptPieces, three for each SM).
constexpr int kPromptPieces = 444, kPromptMostPieces = 8, kPieceSteps = 16;
static_assert(256 + kPromptPieces * 8 <= kPagedHead, "the counts of finished pieces lie in the head");
inline int prompt_pack(const PagedShape& s, int n_heads) {
  const int group = n_heads / s.kv, pack = group & -group;
  return pack < 128 ? pack : 128;
}
struct PromptPlan {
  long long blocks;
  int pieces;
  size_t total;
};
inline PromptPlan prompt_plan(const PagedShape& s, int n_heads, int n_lanes, int n_rows) {
  const int pack = prompt_pack(s, n_heads), pieces = s.max_len() / (kPieceSteps * 64);
  PromptPlan w;
  w.blocks = ((long long)n_rows / (256 / pack) + n_lanes) * (n_heads / pack);  // at least the lanes' blocks
  w.pieces = pieces < 1 ? 1 : pieces > kPromptMostPieces ? kPromptMostPieces : pieces;
  w.total = kPagedHead + (w.pieces > 1 ? (size_t)kPromptPieces * 2 * 128 * (s.hd + 2) * 4 : 0);
  return w;
}
struct PagedOpsWorkspace {
  size_t count_off, moves_off, list_off, total;
};
inline PagedOpsWorkspace paged_ops_workspace(const PagedShape& s) {
  PagedOpsWorkspace w;
  w.count_off = kPagedHead;
  w.moves_off = kPagedHead + 256;
  w.list_off = align256(w.moves_off + (size_t)s.n_pages * 8);
  w.total = align256(w.list_off + (size_t)s.n_pages * 4);
  return w;
}

struct PagedDecodeArgs {
  PagedShape s;
  PagedBufs c;
  int layer, n_heads, n_lanes;
  const void* q;
  int64_t q_stride;
  const int32_t* kv_len;
  const int32_t* seqs;
  float scale;
  void* out;
  uint8_t* ws;
  PagedWorkspace wl;
};
struct PagedPromptArgs {
  PagedShape s;
  PagedBufs c;
  int layer, n_heads, n_lanes, n_rows;
  const void* q;
  int64_t q_stride;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* seqs;
  float scale;
  void* out;
  uint8_t* ws;
  PromptPlan plan;
};

cudaError_t launch_paged_append(const PagedShape& s, const PagedBufs& c, int layer, const void* k_rows, int64_t k_stride,
                                const void* v_rows, int64_t v_stride, int n_rows, const int32_t* cu_rows,
                                const int32_t* start_pos, const int32_t* seqs, int n_lanes, uint32_t* status,
                                cudaStream_t st);                                       // k_paged_append.cu
cudaError_t launch_paged_decode(const PagedDecodeArgs& a, cudaStream_t st);             // k_paged_decode.cu
cudaError_t launch_paged_prompt(const PagedPromptArgs& a, cudaStream_t st);             // k_paged_prompt.cu
// k_paged_pages.cu
cudaError_t launch_paged_copy(const PagedShape& s, const PagedBufs& c, const int32_t* src, const int32_t* dst, int n,
                              uint8_t* ws, cudaStream_t st);
cudaError_t launch_paged_fork(const PagedShape& s, const PagedBufs& c, const int32_t* src, const int32_t* dst,
                              const int32_t* n_tokens, int n, uint8_t* ws, cudaStream_t st);
cudaError_t launch_paged_reserve(const PagedShape& s, const PagedBufs& c, const int32_t* seqs, const int32_t* ctx_len,
                                 const int32_t* n_new, int n, uint8_t* ws, cudaStream_t st);
cudaError_t launch_paged_free(const PagedShape& s, const PagedBufs& c, const int32_t* seqs, const int32_t* keep, int n,
                              uint8_t* ws, cudaStream_t st);
cudaError_t launch_paged_compact(const PagedShape& s, const PagedBufs& c, int32_t* n_live, uint8_t* ws,
                                 cudaStream_t st);

}  // namespace tl
