// Attention of one new token per lane over the paged K/V cache (tl_paged_attn_decode), sm_100a.
//
// Per lane b and query head h of K/V head g: out = sum_c p_c v_c / sum_c p_c with
// p_c = exp2((q . k_c - m) scale log2 e), m the running maximum: one pass over K and V.
//
// What bounds it: every byte of K and V is read once for the whole group of query heads that share
// the K/V head, 2 x group operations per byte, far below the ridge: HBM.  So the design is about
// bytes in flight.  A lane's positions are cut into splits (paged_internal.cuh); one CTA of four warps
// takes one (lane, split, K/V head, tile of 16 query heads).  Each warp works alone on units of 16
// positions (a unit never crosses a page) with a ring of its own, filled by 16-byte asynchronous
// copies, so the loop has no block barrier; the four running (max, sum, out) states are joined at
// the end in shared memory.  The products are m16n8k16 matrix instructions: 16 query heads x 16
// positions; at 16 rows per K/V byte the matrix work is a few percent of their rate, and their
// operands come from registers, without the tensor-memory round trips of tcgen05 that bound
// the store-h streaming kernel.  Measured: 32 lanes of 4097 positions, 16 heads x 128, 172 us a launch, 6.2
// TB/s (0.96 of a copy's bandwidth); 48 lanes of 0 to 8192, 32 heads over 8, 139 us, 5.9 TB/s; one lane of 60001
// over 2 K/V heads 16.5 us, of which 8 are the stream and 4 the loads of its length, its pages and its first rows,
// one behind the other.
//
// Precision: scores, statistics and sums in FP32; p is rounded to the cache's type for the second
// product (half a step, 2^-11 or 2^-8 relative, the rounding that the output itself has, and in FP16 at
// least 2^-40 of the split's largest), its sum is of the unrounded p.
#include <cuda_bf16.h>

#include "paged_internal.cuh"
#include "tc_ptx.cuh"

namespace tl {
namespace {

constexpr int kWarps = 4;
constexpr int kDecThreads = 32 * kWarps;
constexpr int kUnit = 16;       // positions a warp takes at a time
constexpr int kRing = 96 << 10;  // shared memory of a CTA's rings: two CTAs per SM
constexpr float kLog2e = 1.4426950408889634f;
// FP16's exponents end soon: p is held 2^15 times as large (at most 2^15 of 65504), and the weights that FP16 spaces
// 2^-24 apart are those below 2^-29 of the largest instead of 2^-14.  Sums and outputs carry the factor alike.  BF16 has
// FP32's exponents and needs none.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 15.0f;

struct DecodeParams {
  PagedShape s;
  const uint16_t* k;  // the layer's
  const uint16_t* v;
  const int32_t* table;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* kv_len;
  const int32_t* seqs;
  uint16_t* out;
  float* ml;   // [lanes][heads][s_max][2]
  float* acc;  // [lanes][heads][s_max][hd]
  uint32_t* status;
  float scale2;  // scale * log2 e
  int n_heads, group, head_tiles, n_lanes, s_max, target, rows;
};

// Positions lane b attends, or -1 for a lane that is out of range.
__device__ __forceinline__ int lane_len(const DecodeParams& p, int b, int* seq) {
  const int s = p.seqs ? p.seqs[b] : b, n = p.kv_len[b];
  *seq = s;
  return s >= 0 && s < p.s.max_seqs && n >= 0 && n <= p.s.max_len() ? n : -1;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (BF16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// First split of every lane, by all threads: prefix[b] for b < n_lanes, prefix[n_lanes] = all.
__device__ void lane_splits(const DecodeParams& p, int* prefix) {
  __shared__ int part[kWarps];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int done = 0;
  for (int base = 0; base < p.n_lanes; base += kDecThreads) {
    const int b = base + t;
    int n = 0;
    if (b < p.n_lanes) {
      int seq;
      const int len = lane_len(p, b, &seq);
      if (len < 0) {
        if (blockIdx.x == 0) atomicOr(p.status, kStatusRange);
      } else {
        n = paged_splits(len, p.target, p.rows);
      }
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int before = done;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += part[w];
      done += part[w];
    }
    if (b < p.n_lanes) prefix[b] = before + incl - n;
    __syncthreads();
  }
  if (t == 0) prefix[p.n_lanes] = done;
  __syncthreads();
}

template <int HD, bool BF16>
__global__ void __launch_bounds__(kDecThreads, 2) paged_decode_kernel(const DecodeParams p) {
  constexpr int kRowBytes = HD * 2, kHalf = kUnit * kRowBytes, kStageBytes = 2 * kHalf;  // K, then V
  constexpr int kStages = kRing / kWarps / kStageBytes;
  constexpr int kKSteps = HD / 16, kChunks = HD / 8;  // 16-byte chunks of a row
  constexpr int kCopies = kUnit * kChunks / 32;       // 16-byte copies a lane makes for a unit's K (and V)
  static_assert(kStages >= 3, "a ring holds one unit in use and two on their way");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int prefix[kPagedMaxLanes + 1];
  __shared__ float wm[kWarps][16], wl[kWarps][16];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  lane_splits(p, prefix);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* ring = smem + warp * (kRing / kWarps);
  const uint32_t ring_addr = ptx::smem_addr(ring);
  const PagedShape& s = p.s;
  const int tiles = s.kv * p.head_tiles, log_page = 31 - __clz(s.page);
  const int items = prefix[p.n_lanes] * tiles;  // at most 1024 lanes x s_max splits x tiles: checked on the host

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    // tiles of one split are neighbours: they are the same pages
    const int tile = item % tiles, gs = item / tiles;
    int b = 0, hi = p.n_lanes;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (prefix[mid] <= gs)
        b = mid;
      else
        hi = mid;
    }
    const int split = gs - prefix[b], n_splits = prefix[b + 1] - prefix[b];
    const int kvh = tile / p.head_tiles, h0 = kvh * p.group + (tile % p.head_tiles) * 16;
    const int n_rows = min(16, (kvh + 1) * p.group - h0);  // query heads of the tile
    int seq;
    const int len = lane_len(p, b, &seq);
    const int per = paged_split_rows(len, p.target, p.rows);
    const int c0 = split * per, c1 = min(len, c0 + per);
    const int units = c1 > c0 ? (c1 - c0 + kUnit - 1) / kUnit : 0;
    const int my_units = units > warp ? (units - warp + kWarps - 1) / kWarps : 0;  // units warp, warp + 4, ...
    const int32_t* row = p.table + (size_t)seq * s.max_pages;

    // pages of this warp's next 32 units, one per lane
    int pages = -1;
    auto load_pages = [&](int i0) {
      const int i = i0 + lane;
      pages = -1;
      if (i < my_units) {
        const int pg = row[(c0 + (warp + i * kWarps) * kUnit) >> log_page];
        if (pg >= 0 && pg < s.n_pages)
          pages = pg;
        else
          atomicOr(p.status, kStatusRange);
      }
    };
    auto issue = [&](int i) {  // unit i of this warp into its stage
      if (i < my_units) {
        if ((i & 31) == 0) load_pages(i);
        const int pg = __shfl_sync(0xffffffffu, pages, i & 31);
        const int pos = c0 + (warp + i * kWarps) * kUnit;
        const size_t at = ((size_t)(pg < 0 ? 0 : pg) * s.kv + kvh) * s.block_elems() + (size_t)(pos & (s.page - 1)) * HD;
        const uint32_t dst = ring_addr + (i % kStages) * kStageBytes;
#pragma unroll
        for (int k = 0; k < kCopies; ++k) {
          const int e = k * 32 + lane, r = e / kChunks, ch = e % kChunks;
          const uint32_t to = dst + r * kRowBytes + ((ch ^ (r & 7)) << 4);
          const bool valid = pg >= 0 && pos + r < c1;  // rows past the end are zeros: 0 x NaN would spoil the sum
          cp_async16(to, p.k + at + (size_t)r * HD + ch * 8, valid);
          cp_async16(to + kHalf, p.v + at + (size_t)r * HD + ch * 8, valid);
        }
      }
      cp_commit();
    };
    // whether unit i has a page, known when it was issued: kept as one bit per stage
    uint32_t no_page = 0;
    auto issue_noted = [&](int i) {
      issue(i);
      if (i < my_units) {
        const bool none = __shfl_sync(0xffffffffu, pages, i & 31) < 0;
        no_page = (no_page & ~(1u << (i % kStages))) | ((none ? 1u : 0u) << (i % kStages));
      }
    };

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue_noted(i);

    // the queries as the first product's A operand; heads past the tile's are zeros
    uint32_t qf[kKSteps][4];
    {
      const int g = lane >> 2, cc = (lane & 3) * 2;
      const uint16_t* q0 = p.q + (size_t)b * p.q_stride + (size_t)h0 * HD;
#pragma unroll
      for (int k = 0; k < kKSteps; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = g + (i & 1) * 8;
          qf[k][i] = r < n_rows ? *reinterpret_cast<const uint32_t*>(q0 + (size_t)r * HD + k * 16 + cc + (i >> 1) * 8) : 0u;
        }
    }
    float o[HD / 8][4];
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // rows lane / 4 and + 8; l: this lane's columns

    // ldmatrix addresses inside a stage.  K: matrices (positions 0-7 | 8-15) x (values 0-7 | 8-15) of a
    // 16-value step; V, transposed: the same four, which gives the B operand of 8 + 8 output values.
    const int mr = lane & 7, mi = lane >> 3;
    const int k_row = mr + (mi >> 1) * 8, k_ch = mi & 1;
    const int v_row = mr + (mi & 1) * 8, v_ch = mi >> 1;
    for (int i = 0; i < my_units; ++i) {
      cp_wait<kStages - 2>();
      __syncwarp();
      const uint32_t st = ring_addr + (i % kStages) * kStageBytes;
      float sc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int k = 0; k < kKSteps; ++k) {
        uint32_t f[4];
        ldsm4(st + k_row * kRowBytes + (((2 * k + k_ch) ^ (k_row & 7)) << 4), f);
        mma16816<BF16>(sc[0], qf[k], f[0], f[1]);
        mma16816<BF16>(sc[1], qf[k], f[2], f[3]);
      }
      const int left = (no_page >> (i % kStages)) & 1 ? 0 : c1 - (c0 + (warp + i * kWarps) * kUnit);
      if (left < kUnit) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (nb * 8 + (lane & 3) * 2 + (j & 1) >= left) sc[nb][j] = -INFINITY;
      }
      float corr[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        x = fmaxf(x, m[r]);
        const float base = x == -INFINITY ? 0.0f : x * p.scale2;  // nothing attended yet: every p is exp2(-inf) = 0
        const float lift = kLift<BF16> - base;
        corr[r] = ex2(m[r] * p.scale2 - base);
        if (m[r] == x) corr[r] = 1.0f;
        m[r] = x;
        float sum = 0.0f;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float e = ex2(fmaf(sc[nb][2 * r + j], p.scale2, lift));
            sc[nb][2 * r + j] = e;
            sum += e;
          }
        l[r] = fmaf(l[r], corr[r], sum);
      }
      if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
        for (int n = 0; n < HD / 8; ++n) {
          o[n][0] *= corr[0];
          o[n][1] *= corr[0];
          o[n][2] *= corr[1];
          o[n][3] *= corr[1];
        }
      }
      const uint32_t pf[4] = {pack16<BF16>(sc[0][0], sc[0][1]), pack16<BF16>(sc[0][2], sc[0][3]),
                              pack16<BF16>(sc[1][0], sc[1][1]), pack16<BF16>(sc[1][2], sc[1][3])};
#pragma unroll
      for (int n = 0; n < HD / 16; ++n) {
        uint32_t f[4];
        ldsm4_t(st + kHalf + v_row * kRowBytes + (((2 * n + v_ch) ^ (v_row & 7)) << 4), f);
        mma16816<BF16>(o[2 * n], pf, f[0], f[1]);
        mma16816<BF16>(o[2 * n + 1], pf, f[2], f[3]);
      }
      __syncwarp();  // every lane has read the stage that the next copy overwrites
      issue_noted(i + kStages - 1);
    }
    cp_wait<0>();
    __syncwarp();

    // join the four warps: each leaves its sums in its own ring, then the threads share the outputs
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if ((lane & 3) == 0) {
        wm[warp][(lane >> 2) + 8 * r] = m[r];
        wl[warp][(lane >> 2) + 8 * r] = l[r];
      }
    }
    float* mine = reinterpret_cast<float*>(ring);  // [16][HD]
#pragma unroll
    for (int n = 0; n < HD / 8; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        *reinterpret_cast<float2*>(mine + ((lane >> 2) + 8 * r) * HD + n * 8 + (lane & 3) * 2) =
            make_float2(o[n][2 * r], o[n][2 * r + 1]);
    __syncthreads();
    for (int e = threadIdx.x; e < n_rows * (HD / 4); e += kDecThreads) {
      const int r = e / (HD / 4), d = e % (HD / 4) * 4;
      float mx = wm[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, wm[w][r]);
      float sum = 0.0f;
      float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = wm[w][r] == -INFINITY ? 0.0f : ex2((wm[w][r] - mx) * p.scale2);
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * (kRing / kWarps)) + r * HD + d);
        sum = fmaf(wl[w][r], f, sum);
        a.x = fmaf(x.x, f, a.x);
        a.y = fmaf(x.y, f, a.y);
        a.z = fmaf(x.z, f, a.z);
        a.w = fmaf(x.w, f, a.w);
      }
      const size_t head = (size_t)b * p.n_heads + h0 + r;
      if (n_splits == 1) {
        const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
        *reinterpret_cast<uint2*>(p.out + head * HD + d) =
            make_uint2(pack16<BF16>(a.x * inv, a.y * inv), pack16<BF16>(a.z * inv, a.w * inv));
      } else {
        const size_t part = head * p.s_max + split;
        *reinterpret_cast<float4*>(p.acc + part * HD + d) = a;
        if (d == 0) *reinterpret_cast<float2*>(p.ml + part * 2) = make_float2(mx, sum);
      }
    }
    __syncthreads();
  }
}

// Joins the n splits of one (lane, query head), COLS of its values: a thread four values of every kAtOnce-th split,
// eight loads in flight.  (The last CTA of a lane joining its splits inside the kernel above was measured instead: the
// fence and the counter's round trip stand at the end of every split, 10.1 us a call against 8.9 at one lane of
// 2049, 193 us against 184 at 32 lanes of 4097.)
constexpr int kJoinThreads = 256;
template <int HD, int COLS, bool BF16>
__device__ __forceinline__ void join_splits(const DecodeParams& p, int n) {
  constexpr int kLanes = COLS / 4, kAtOnce = kJoinThreads / kLanes, kWindow = kAtOnce * 8;  // splits a round
  __shared__ float4 part[kAtOnce][kLanes];
  __shared__ float weight[kWindow], psum[kJoinThreads / 32], pmax[kJoinThreads / 32];
  const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x, col = blockIdx.z * COLS;
  const size_t first = ((size_t)b * p.n_heads + h) * p.s_max;
  const float2* ml = reinterpret_cast<const float2*>(p.ml) + first;
  const int d = t % kLanes, g = t / kLanes;
  float4 a = make_float4(0, 0, 0, 0);
  float sum = 0.0f, top = -INFINITY;  // of this thread's splits; of all splits so far
  for (int i0 = 0; i0 < n; i0 += kWindow) {
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * kAtOnce + g;
      if (i < n) x[k] = *reinterpret_cast<const float4*>(p.acc + (first + i) * HD + col + d * 4);
    }
    const float2 s = t < kWindow && i0 + t < n ? ml[i0 + t] : make_float2(-INFINITY, 0.0f);
    float mx = s.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((t & 31) == 0) pmax[t >> 5] = mx;
    __syncthreads();
    mx = top;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) mx = fmaxf(mx, pmax[w]);
    const float old = top == -INFINITY ? 0.0f : ex2((top - mx) * p.scale2);
    top = mx;
    const float f = s.x == -INFINITY ? 0.0f : ex2((s.x - mx) * p.scale2);
    if (t < kWindow) weight[t] = f;
    sum = fmaf(sum, old, s.y * f);
    a = make_float4(a.x * old, a.y * old, a.z * old, a.w * old);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = k * kAtOnce + g;
      if (i0 + i < n) {
        a.x = fmaf(x[k].x, weight[i], a.x);
        a.y = fmaf(x[k].y, weight[i], a.y);
        a.z = fmaf(x[k].z, weight[i], a.z);
        a.w = fmaf(x[k].w, weight[i], a.w);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((t & 31) == 0) psum[t >> 5] = sum;
  part[g][d] = a;
  __syncthreads();
  if (t < kLanes) {
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) sum += psum[w];
    a = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float4 y = part[i][d];
      a.x += y.x;
      a.y += y.y;
      a.z += y.z;
      a.w += y.w;
    }
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    *reinterpret_cast<uint2*>(p.out + ((size_t)b * p.n_heads + h) * HD + col + d * 4) =
        make_uint2(pack16<BF16>(a.x * inv, a.y * inv), pack16<BF16>(a.z * inv, a.w * inv));
  }
}

// More than kJoinWide splits are joined by HD / 32 CTAs, 32 values each, a round of 256 splits then: one lane of 60000
// over 148 splits 20.6 -> 19.5 us a call, of 40000 over 74 23.3 -> 21.8; with fewer, one CTA takes them in a round as it
// is (37 splits the same, 48 lanes of up to 8 splits 150 us against 136).  By the lane's own splits, so that its bits
// depend on nothing else.
constexpr int kJoinWide = 64;
template <int HD, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const DecodeParams p) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  int seq;
  const int len = lane_len(p, blockIdx.y, &seq), n = len < 0 ? 0 : paged_splits(len, p.target, p.rows);
  if (n <= 1) return;  // a single split wrote the output itself
  if (n > kJoinWide)
    join_splits<HD, 32, BF16>(p, n);
  else if (blockIdx.z == 0)
    join_splits<HD, HD, BF16>(p, n);
}

template <int HD, bool BF16>
cudaError_t launch_as(const DecodeParams& p, cudaStream_t st) {
  int limit = 0;
  cudaError_t e = dyn_smem_limit((const void*)paged_decode_kernel<HD, BF16>, &limit);
  if (e != cudaSuccess) return e;
  if (kRing > limit) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  const long long items = (long long)p.n_lanes * p.s_max * p.s.kv * p.head_tiles;
  cfg.gridDim = dim3((unsigned)(items < kPagedSlots ? items : kPagedSlots));
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = kRing;
  profile_stream_begin(st);
  e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<HD, BF16>, p);
  profile_stream_end(st);
  count_launch();
  if (e != cudaSuccess) return e;
  if (p.s_max > 1) {
    cfg.gridDim = dim3((unsigned)p.n_heads, (unsigned)p.n_lanes, p.s_max > kJoinWide ? HD / 32 : 1);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, paged_join_kernel<HD, BF16>, p);
    count_launch();
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, cudaStream_t st) {
  const PagedShape& s = a.s;
  const size_t off = (size_t)a.layer * s.layer_elems();
  const int group = a.n_heads / s.kv;
  DecodeParams p{s,
                 a.c.k + off,
                 a.c.v + off,
                 a.c.table,
                 (const uint16_t*)a.q,
                 a.q_stride,
                 a.kv_len,
                 a.seqs,
                 (uint16_t*)a.out,
                 (float*)(a.ws + a.wl.ml_off),
                 (float*)(a.ws + a.wl.acc_off),
                 (uint32_t*)a.ws,
                 a.scale * kLog2e,
                 a.n_heads,
                 group,
                 (group + 15) / 16,
                 a.n_lanes,
                 a.wl.s_max,
                 a.wl.target,
                 a.wl.rows};
  if (s.hd == 64) return s.dtype == TL_KV_BF16 ? launch_as<64, true>(p, st) : launch_as<64, false>(p, st);
  return s.dtype == TL_KV_BF16 ? launch_as<128, true>(p, st) : launch_as<128, false>(p, st);
}

}  // namespace tl
