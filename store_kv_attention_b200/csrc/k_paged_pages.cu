// Operations on the pages of the paged K/V cache: copy, fork, reserve, free, compact.
//
// Copy, reserve and compact come down to a list of moves (source page, destination page), planned by
// one block from the table and the counts (a few scans over lists that lie in L2: latency bound),
// then carried out on every layer's K and V by all SMs (2 x moves x layers x 2 x page bytes: HBM
// bound).  No destination of a plan is a source of it, so the moves need no order.  Pages are taken
// in the order of prefix sums, never of atomics, so results do not depend on scheduling.  Measured: compaction
// of 8192 pages of 4 layers (8 heads x 128 x 16 positions), 1.06 GB moved in 172 us, 6.2 TB/s, its plan 11 us;
// room for one token for 48 forks, plan 9.7 us, copies 7.2.
#include "paged_internal.cuh"
#include "tc_ptx.cuh"

namespace tl {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveChunk = kMoveThreads * 4;  // 16-byte words a block moves at a time

struct Plan {
  uint32_t* status;
  int32_t* count;  // moves
  int2* moves;
  int32_t* list;   // one word per page
};
Plan plan_of(const PagedShape& s, uint8_t* ws) {
  const PagedOpsWorkspace w = paged_ops_workspace(s);
  return Plan{(uint32_t*)ws, (int32_t*)(ws + w.count_off), (int2*)(ws + w.moves_off), (int32_t*)(ws + w.list_off)};
}

// Exclusive sum of x over the block's threads in thread order; *total receives the sum.  (T: int, or long long
// for several counts side by side.)
template <typename T>
__device__ T block_scan(T x, T* total) {
  __shared__ T part[kPlanThreads / 32];
  __shared__ T sum;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const T p = part[lane];
    T q = p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, q, o);
      if (lane >= o) q += y;
    }
    part[lane] = q - p;
    if (lane == 31) sum = q;
  }
  __syncthreads();
  const T before = part[warp];
  *total = sum;
  __syncthreads();
  return before + incl - x;
}

// The counts of 16 pages from p0 on (a multiple of 4; refs is 256-byte aligned); -1 from `end` on.
__device__ __forceinline__ void load_refs(const int32_t* refs, int p0, int end, int* r) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    if (p0 + i + 3 < end) {
      const int4 x = *reinterpret_cast<const int4*>(refs + p0 + i);
      r[i] = x.x, r[i + 1] = x.y, r[i + 2] = x.z, r[i + 3] = x.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) r[i + k] = p0 + i + k < end ? refs[p0 + i + k] : -1;
    }
  }
}

// The first `most` free pages, lowest first, into list; returns how many pages are free, counted until there are
// `most`.
__device__ int free_pages_of(const int32_t* refs, int n_pages, int most, int32_t* list) {
  int seen = 0;
  for (int base = 0; base < n_pages && seen < most; base += kPlanThreads * 16) {
    const int p0 = base + threadIdx.x * 16;
    int r[16], n = 0;
    load_refs(refs, p0, n_pages, r);
#pragma unroll
    for (int i = 0; i < 16; ++i) n += p0 + i < n_pages && r[i] <= 0;
    int total;
    int rank = seen + block_scan(n, &total);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (p0 + i < n_pages && r[i] <= 0) {
        if (rank < most) list[rank] = p0 + i;
        ++rank;
      }
    seen += total;
  }
  return seen;
}

// Carries out the plan's moves.  remap: the table's entries follow (list[old page] = new page for the
// pages that moved, the others keep theirs: moved pages are those at or above *bound).
__global__ void __launch_bounds__(kMoveThreads)
    paged_move_kernel(PagedShape s, PagedBufs c, Plan plan, bool remap) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int n = *plan.count;
  const size_t words = s.page_elems() / 8;
  const int chunks = (int)((words + kMoveChunk - 1) / kMoveChunk);
  const long long items = (long long)n * s.layers * 2 * chunks;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int chunk = (int)(it % chunks);
    const long long t = it / chunks;
    const bool is_v = t & 1;
    const int layer = (int)((t >> 1) % s.layers), m = (int)((t >> 1) / s.layers);
    const int2 mv = plan.moves[m];
    uint4* pool = reinterpret_cast<uint4*>((is_v ? c.v : c.k) + (size_t)layer * s.layer_elems());
    const uint4* src = pool + (size_t)mv.x * words;
    uint4* dst = pool + (size_t)mv.y * words;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t at = (size_t)chunk * kMoveChunk + i * kMoveThreads + threadIdx.x;
      if (at < words) x[i] = src[at];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t at = (size_t)chunk * kMoveChunk + i * kMoveThreads + threadIdx.x;
      if (at < words) dst[at] = x[i];
    }
  }
  if (!remap || n == 0) return;
  const int bound = plan.count[1];
  const size_t entries = (size_t)s.max_seqs * s.max_pages;
  for (size_t e = (size_t)blockIdx.x * kMoveThreads + threadIdx.x; e < entries; e += (size_t)gridDim.x * kMoveThreads) {
    const int p = c.table[e];
    if (p >= bound && p < s.n_pages) {
      const int to = plan.list[p];
      if (to >= 0) c.table[e] = to;
    }
  }
}

// ---------------------------------------------------------------- copy
__global__ void __launch_bounds__(kPlanThreads)
    paged_copy_plan_kernel(PagedShape s, Plan plan, const int32_t* src, const int32_t* dst, int n) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  // list[page] = the first pair that names the page as its destination, n for a page that none does
  // (only the words of pages in the lists are used)
  auto in_pool = [&](int p) { return p >= 0 && p < s.n_pages; };
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    if (in_pool(src[i])) plan.list[src[i]] = n;
    if (in_pool(dst[i])) plan.list[dst[i]] = n;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (in_pool(dst[i])) atomicMin(&plan.list[dst[i]], i);
  __syncthreads();
  int made = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    bool ok = i < n && in_pool(src[i]) && in_pool(dst[i]);
    // atomics act in L2: read past this SM's L1
    if (ok) ok = __ldcg(&plan.list[dst[i]]) == i && __ldcg(&plan.list[src[i]]) == n;
    if (i < n && !ok) atomicOr(plan.status, kStatusRange);
    int total;
    const int at = made + block_scan<int>(ok, &total);
    if (ok) plan.moves[at] = make_int2(src[i], dst[i]);
    made += total;
  }
  if (threadIdx.x == 0) plan.count[0] = made;
}

// ---------------------------------------------------------------- fork
constexpr int kRowThreads = 256;

// One block per fork.  dst rows that another fork reads are refused, so no block reads what another writes.
__global__ void __launch_bounds__(kRowThreads)
    paged_fork_kernel(PagedShape s, PagedBufs c, const int32_t* src, const int32_t* dst, const int32_t* n_tokens, int n,
                      uint32_t* status) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int i = blockIdx.x, a = src[i], d = dst[i], len = n_tokens[i];
  bool ok = a >= 0 && a < s.max_seqs && d >= 0 && d < s.max_seqs && len >= 0 && len <= s.max_len();
  if (ok)
    for (int k = threadIdx.x; k < n; k += kRowThreads)
      if (dst[k] == a || (k < i && dst[k] == d)) ok = false;
  const int pages = ok ? (int)(((long long)len + s.page - 1) / s.page) : 0;
  const int32_t* from = c.table + (size_t)(ok ? a : 0) * s.max_pages;
  int32_t* to = c.table + (size_t)(ok ? d : 0) * s.max_pages;
  if (ok)
    for (int j = threadIdx.x; j < s.max_pages; j += kRowThreads) {
      if (to[j] >= 0) ok = false;
      if (j < pages) {
        const int p = from[j];
        if (p < 0 || p >= s.n_pages) ok = false;
      }
    }
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) atomicOr(status, kStatusRange);
    return;
  }
  for (int j = threadIdx.x; j < pages; j += kRowThreads) {
    const int p = from[j];
    to[j] = p;
    atomicAdd(&c.refs[p], 1);
  }
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(kRowThreads)
    paged_free_kernel(PagedShape s, PagedBufs c, const int32_t* seqs, const int32_t* keep, uint32_t* status) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int q = seqs[blockIdx.x], kept = keep ? keep[blockIdx.x] : 0;
  if (q < 0 || q >= s.max_seqs || kept < 0) {
    if (threadIdx.x == 0) atomicOr(status, kStatusRange);
    return;
  }
  const long long from = ((long long)kept + s.page - 1) / s.page;
  int32_t* row = c.table + (size_t)q * s.max_pages;
  // the exchange gives each entry to one block when a sequence is listed twice
  for (long long j = from + threadIdx.x; j < s.max_pages; j += kRowThreads) {
    const int p = atomicExch(&row[j], -1);
    if (p >= 0 && p < s.n_pages) atomicSub(&c.refs[p], 1);
  }
}

// ---------------------------------------------------------------- reserve
// Candidates are the entries that the listed sequences write, in list order: flattened, so that one
// long prompt and a thousand single tokens spread over the threads alike.  Two passes over them (does
// the entry need a page; which one does it get) around the list of free pages.
__global__ void __launch_bounds__(kPlanThreads)
    paged_reserve_plan_kernel(PagedShape s, PagedBufs c, Plan plan, const int32_t* seqs, const int32_t* ctx_len,
                              const int32_t* n_new, int n) {
  __shared__ int start[kPagedMaxLanes + 1];  // first candidate of each sequence
  __shared__ int first[kPagedMaxLanes];      // its first entry, or -1: refused
  __shared__ __align__(16) int ids[kPagedMaxLanes];
  __shared__ int n_served;                   // sequences that the free pages cover
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int t = threadIdx.x;
  int seq = -1, ctx = 0, add = 0;
  if (t < n) {
    seq = seqs[t];
    ctx = ctx_len[t];
    add = n_new[t];
    ids[t] = seq;
  }
  __syncthreads();
  int span = 0;
  if (t < n) {
    bool ok = seq >= 0 && seq < s.max_seqs && ctx >= 0 && add >= 0 && (long long)ctx + add <= s.max_len();
#pragma unroll 4
    for (int k = 0; k < t; k += 4) {
      const int4 x = *reinterpret_cast<const int4*>(ids + k);
      ok = ok && x.x != seq && (k + 1 >= t || x.y != seq) && (k + 2 >= t || x.z != seq) && (k + 3 >= t || x.w != seq);
    }
    if (!ok) atomicOr(plan.status, kStatusRange);
    first[t] = ok ? ctx / s.page : 0;
    if (ok && add > 0) span = (ctx + add - 1) / s.page - ctx / s.page + 1;
  }
  int total;
  const int at = block_scan(span, &total);
  if (t < n) start[t] = at;
  if (t == 0) {
    start[n] = total;
    n_served = n;
  }
  __syncthreads();

  // entry of candidate i: its sequence's place in the list (the last one that starts at or before i)
  auto find = [&](int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= i)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };
  // whether the entry needs a page of its own; *was = the page it names
  auto needs = [&](int k, int i, int* was) {
    const int p = c.table[(size_t)ids[k] * s.max_pages + first[k] + i - start[k]];
    *was = p;
    return p < 0 || p >= s.n_pages || c.refs[p] > 1;
  };
  // pass 1: how many pages are needed
  int needed = 0;
  for (int base = 0; base < total; base += kPlanThreads) {
    const int i = base + t;
    int was;
    needed += __syncthreads_count(i < total && needs(find(i), i, &was));
  }
  // the lowest free pages
  const int free_pages = free_pages_of(c.refs, s.n_pages, needed, plan.list);
  // too few: the first sequence whose need, with those before it, passes them
  if (free_pages < needed) {
    int before = 0;
    for (int base = 0; base < total; base += kPlanThreads) {
      const int i = base + t;
      int was, sum;
      const int k = i < total ? find(i) : 0;
      const bool need = i < total && needs(k, i, &was);
      const int rank = before + block_scan<int>(need, &sum);
      if (need && rank >= free_pages) atomicMin(&n_served, k);
      before += sum;
    }
    if (t == 0) atomicOr(plan.status, kStatusFull);
  }
  __syncthreads();
  const int end = n_served == n ? total : start[n_served];
  // pass 2: the k-th need gets the k-th free page.  Counts change only after every need was decided;
  // replaced pages are noted in moves, those without rows to keep behind the ones that are copied.
  int given = 0, copies = 0, drops = 0;
  for (int base = 0; base < end; base += kPlanThreads) {
    const int i = base + t;
    int was = -1, k = 0;
    bool need = false;
    if (i < end) {
      k = find(i);
      need = needs(k, i, &was);
    }
    const bool shared = need && was >= 0 && was < s.n_pages;
    const int j = i < end ? first[k] + i - start[k] : 0;
    const bool copy = shared && i == start[k] && (ctx_len[k] % s.page) != 0;  // only its first entry holds rows before ctx_len
    // needs, copies and drops counted side by side
    long long sum;
    const long long at = block_scan<long long>((long long)need | (long long)copy << 20 | (long long)(shared && !copy) << 40, &sum);
    constexpr int kMask = (1 << 20) - 1;
    const int rank = given + (int)(at & kMask), mc = (int)(at >> 20 & kMask), md = (int)(at >> 40);
    const int n_copy = (int)(sum >> 20 & kMask), n_drop = (int)(sum >> 40);
    given += (int)(sum & kMask);
    const int to = need ? plan.list[rank] : -1;
    if (copy) plan.moves[copies + mc] = make_int2(was, to);
    if (shared && !copy) plan.moves[s.n_pages - 1 - (drops + md)] = make_int2(was, to);
    copies += n_copy;
    drops += n_drop;
    if (need) c.table[(size_t)ids[k] * s.max_pages + j] = to;
  }
  __syncthreads();
  for (int i = t; i < given; i += kPlanThreads) c.refs[plan.list[i]] = 1;
  for (int i = t; i < copies; i += kPlanThreads) atomicSub(&c.refs[plan.moves[i].x], 1);
  for (int i = t; i < drops; i += kPlanThreads) atomicSub(&c.refs[plan.moves[s.n_pages - 1 - i].x], 1);
  if (t == 0) plan.count[0] = copies;
}

// ---------------------------------------------------------------- compact
__global__ void __launch_bounds__(kPlanThreads)
    paged_compact_plan_kernel(PagedShape s, PagedBufs c, Plan plan, int32_t* n_live) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  int live, mine = 0, r[16];
  for (int base = 0; base < s.n_pages; base += kPlanThreads * 16) {
    load_refs(c.refs, base + threadIdx.x * 16, s.n_pages, r);
#pragma unroll
    for (int i = 0; i < 16; ++i) mine += r[i] > 0;
  }
  block_scan(mine, &live);
  // free pages below `live` and pages in use from there on: as many of the one as of the other
  int holes = 0, movers = 0;
  for (int base = 0; base < s.n_pages; base += kPlanThreads * 16) {
    const int p0 = base + threadIdx.x * 16;
    if (s.n_pages > kPlanThreads * 16) load_refs(c.refs, p0, s.n_pages, r);  // else they are still there
    int h = 0, m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      h += p0 + i < live && r[i] <= 0;
      m += p0 + i >= live && r[i] > 0;
    }
    long long sum;
    const long long at = block_scan<long long>((long long)h | (long long)m << 32, &sum);
    int hole = holes + (int)(at & 0xffffffff), mover = movers + (int)(at >> 32);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int p = p0 + i;
      if (p < live && r[i] <= 0) plan.moves[hole++].y = p;
      if (p >= live && r[i] > 0) plan.moves[mover++].x = p;
      if (p >= live && p < s.n_pages && r[i] <= 0) plan.list[p] = -1;  // for a table that names a page it does not hold
    }
    holes += (int)(sum & 0xffffffff);
    movers += (int)(sum >> 32);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < holes; i += kPlanThreads) {
    const int2 m = plan.moves[i];
    plan.list[m.x] = m.y;
    c.refs[m.y] = c.refs[m.x];
    c.refs[m.x] = 0;
  }
  if (threadIdx.x == 0) {
    plan.count[0] = holes;
    plan.count[1] = live;
    if (n_live) *n_live = live;
  }
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), int grid, int block, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Blocks for at most `moves` moves: no more than they have chunks, and eight on each SM.
cudaError_t launch_moves(const PagedShape& s, const PagedBufs& c, const Plan& plan, long long moves, bool remap,
                         cudaStream_t st) {
  const long long chunks = ((long long)(s.page_elems() / 8) + kMoveChunk - 1) / kMoveChunk;
  const long long items = moves * s.layers * 2 * chunks;
  return launch(paged_move_kernel, (int)(items < 148 * 8 ? items : 148 * 8), kMoveThreads, st, s, c, plan, remap);
}

}  // namespace

cudaError_t launch_paged_copy(const PagedShape& s, const PagedBufs& c, const int32_t* src, const int32_t* dst, int n,
                              uint8_t* ws, cudaStream_t st) {
  const Plan plan = plan_of(s, ws);
  cudaError_t e = launch(paged_copy_plan_kernel, 1, kPlanThreads, st, s, plan, src, dst, n);
  return e != cudaSuccess ? e : launch_moves(s, c, plan, n, false, st);
}

cudaError_t launch_paged_fork(const PagedShape& s, const PagedBufs& c, const int32_t* src, const int32_t* dst,
                              const int32_t* n_tokens, int n, uint8_t* ws, cudaStream_t st) {
  return launch(paged_fork_kernel, n, kRowThreads, st, s, c, src, dst, n_tokens, n, (uint32_t*)ws);
}

cudaError_t launch_paged_reserve(const PagedShape& s, const PagedBufs& c, const int32_t* seqs, const int32_t* ctx_len,
                                 const int32_t* n_new, int n, uint8_t* ws, cudaStream_t st) {
  const Plan plan = plan_of(s, ws);
  cudaError_t e = launch(paged_reserve_plan_kernel, 1, kPlanThreads, st, s, c, plan, seqs, ctx_len, n_new, n);
  return e != cudaSuccess ? e : launch_moves(s, c, plan, n, false, st);  // one copied page per sequence at most
}

cudaError_t launch_paged_free(const PagedShape& s, const PagedBufs& c, const int32_t* seqs, const int32_t* keep, int n,
                              uint8_t* ws, cudaStream_t st) {
  return launch(paged_free_kernel, n, kRowThreads, st, s, c, seqs, keep, (uint32_t*)ws);
}

cudaError_t launch_paged_compact(const PagedShape& s, const PagedBufs& c, int32_t* n_live, uint8_t* ws,
                                 cudaStream_t st) {
  const Plan plan = plan_of(s, ws);
  cudaError_t e = launch(paged_compact_plan_kernel, 1, kPlanThreads, st, s, c, plan, n_live);
  return e != cudaSuccess ? e : launch_moves(s, c, plan, s.n_pages, true, st);
}

}  // namespace tl
