// Causal attention of packed prompts over the paged K/V cache (tl_paged_prompt_attn) on
// 5th-generation tensor cores (tcgen05 + TMEM), sm_100a.
//
// Per (lane, query head): S = Q K^T, P = exp2((S - m) scale log2 e) with m the running row maximum,
// O = P V / rowsum(P), one pass over K and V in tiles of 128 positions.  4 x hd operations per
// attended pair: the tensor pipe bounds long prompts, and next to it the exponentials (16 a clock and
// SM: 1024 clocks per 128 x 128 tile, as many as its two products at hd = 128).
//
// One CTA takes two tiles of 128 query rows.  A row is a (token, head) pair: the Gp heads of one
// K/V head that fit (Gp the largest power of two up to 128 dividing the group) lie next to each
// other, 128 / Gp tokens a tile, so the heads of a group share their K and V tiles and the causal
// edge is only 128 / Gp tokens wide.  Roles:
//   warps 0-3, 4-7  softmax of tile 0 / 1, a thread per row: S from TMEM, maximum, P back into S's
//                   columns as 16-bit values (A operand of the second product), at the end O / sum
//   warp 8          issues the products: S_t(j+1) follows P_t(j) V(j), so that the tensor pipe
//                   works on one tile while the other one's softmax runs
//   warp 9          TMA producer: Q once, K and V tiles through a ring, page by page (a page of one
//                   K/V head is one box per 64 values)
//   warps 10-11     clean the V tiles that hold positions not every row attends: rows past the
//                   cache's end are zeroed (their memory may hold anything) and values that are not
//                   finite are taken out (0 x inf would reach the rows that do not attend them) and
//                   given back in the epilogue to the rows that do
// O is rescaled only when a row's maximum has grown by more than 2^8 in the exponent since the last
// time (P and its sum stay below 2^8 x 128 tiles' worth of FP32): the exponent's base is a free
// choice, and the rescale, a round trip of O through registers, becomes rare.
//
// TMEM (512 columns): S_0 | S_1 (128 columns each; P over the first 64) | O_0 | O_1.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <mutex>

#include "paged_internal.cuh"
#include "tc_ptx.cuh"

namespace tl {
namespace {

using namespace ptx;

constexpr int kPromptThreads = 384;
constexpr int kTile = 128;
constexpr long long kPWait = 4000000000ll;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;  // growth of the maximum, in powers of two, that O is rescaled for

struct PromptParams {
  PagedShape s;
  const uint16_t* v;  // the layer's
  const int32_t* table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* seqs;
  uint16_t* out;
  uint32_t* status;
  float scale2;  // scale * log2 e
  int n_heads, group, pack, n_rows, n_lanes;
};

template <int HD>
struct PromptSmem {
  static constexpr int kOperand = kTile * HD * 2;  // one tile of Q, K or V
  static constexpr int kSlots = HD == 128 ? 4 : 8;
  static constexpr int kBytes = 1024 + (2 + kSlots) * kOperand;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
#define TL_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : TL_R8(v, 0), TL_R8(v, 8), TL_R8(v, 16), TL_R8(v, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two FP32 values in a 64-bit register, for the packed instructions.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
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
template <bool BF16>
__device__ __forceinline__ float unpack16(uint16_t x) {
  if (BF16) return __uint_as_float((uint32_t)x << 16);
  return __half2float(__ushort_as_half(x));
}
// Instruction descriptor of kind::f16 with FP16 or BF16 operands.
template <bool BF16>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, bool b_mn_major) {
  return idesc_f16_f32(M, N, false, b_mn_major) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
}

// What one CTA works on, worked out by warp 0 and shared.
struct Job {
  int lane;        // -1: nothing to do
  int q0, n_q;     // first packed row and number of queries of the lane
  int kv, seq;     // cached positions, sequence
  int tok0;        // first token of the CTA's first tile
};

// Block `blk` of the lanes' blocks of 2 x tq tokens, a lane's last block first (the longest).
__device__ void find_job(const PromptParams& p, int blk, int tq, Job* job) {
  const int lane = threadIdx.x & 31;
  int found = -1, done = 0;
  for (int base = 0; base < p.n_lanes && (found < 0 || blk == 0); base += 32) {
    const int b = base + lane;
    int n = 0, q0 = 0, blocks = 0;
    if (b < p.n_lanes) {
      q0 = p.cu_q[b];
      const int q1 = p.cu_q[b + 1];
      n = q1 - q0;
      if (q0 < 0 || q1 > p.n_rows || n < 0) {
        if (blk == 0) atomicOr(p.status, kStatusRange);
        n = 0;
      }
      blocks = (n + 2 * tq - 1) / (2 * tq);
    }
    int incl = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned has = __ballot_sync(0xffffffffu, blocks > 0 && blk < done + incl && blk >= done + incl - blocks);
    if (has && found < 0) {
      const int l = __ffs(has) - 1;
      found = base + l;
      if (lane == l) {
        const int seq = p.seqs ? p.seqs[b] : b, kv = p.kv_len[b];
        const bool ok = seq >= 0 && seq < p.s.max_seqs && kv >= 0 && kv <= p.s.max_len();
        if (!ok) atomicOr(p.status, kStatusRange);
        *job = Job{ok ? b : -1, q0, n, kv, seq, (done + incl - 1 - blk) * 2 * tq};
      }
    }
    done += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (found < 0 && lane == 0) job->lane = -1;
}

template <int HD, bool BF16>
__global__ void __launch_bounds__(kPromptThreads, 1)
    paged_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const PromptParams p) {
  constexpr int kOperand = PromptSmem<HD>::kOperand, kSlots = PromptSmem<HD>::kSlots, kVSlots = kSlots / 2;
  constexpr uint32_t kIdS = idesc16<BF16>(128, 128, false), kIdO = idesc16<BF16>(128, HD, true);
  static_assert(kSlots % 2 == 0, "V(j) lies in slot 2 (j mod kVSlots) + 1");
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t q_full, full[kSlots], empty[kSlots], s_full[2], p_full[2], o_done[2], near, clean[kVSlots], fin;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, dirty;
  __shared__ Job job;
  uint8_t* base = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* qs = base;                  // two tiles
  uint8_t* ring = base + 2 * kOperand;  // K(0), V(0), K(1), V(1), ...

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedShape& s = p.s;
  pdl_wait();
  const int subs = p.n_heads / p.pack, sub = blockIdx.x % subs, tq = kTile / p.pack;
  const int h0 = sub * p.pack, kvh = h0 / p.group;
  if (warp == 0) find_job(p, blockIdx.x / subs, tq, &job);
  if (threadIdx.x == 32) {
    mbar_init(&q_full, 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 128);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(&near, 1);
    for (int i = 0; i < kVSlots; ++i) mbar_init(&clean[i], 64);
    mbar_init(&fin, 1);
    abort_flag = 0;
    dirty = 0;
    mbar_fence_init();
  }
  __syncthreads();
  if (job.lane < 0) {
    pdl_trigger();
    return;
  }
  const int n_q = job.n_q, kv_len = job.kv, tok0 = job.tok0;
  const int32_t* row = p.table + (size_t)job.seq * s.max_pages;
  // every page of the lane has to be one of the pool
  bool ok = true;
  for (int j = threadIdx.x; j < (kv_len + s.page - 1) / s.page; j += kPromptThreads) {
    const int pg = row[j];
    ok = ok && pg >= 0 && pg < s.n_pages;
  }
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusRange);
    pdl_trigger();
    return;
  }
  if (warp == 8) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base;
  volatile int* abort_p = &abort_flag;
  pdl_trigger();  // TMEM is held

  const int shift = kv_len - n_q;  // position of token 0
  // K/V tiles each query tile needs, by its last token's position
  int n_t[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = tok0 + t * tq, last = min(n_q, first + tq) - 1;
    n_t[t] = first < n_q && shift + last >= 0 ? (shift + last) / kTile + 1 : 0;
  }
  const int n = max(n_t[0], n_t[1]);
  const int dirty_from = max(0, shift + tok0 + 1) / kTile;  // first tile with positions that not every row attends
  int loads = 0;                                            // ring loads issued (producer warp)
  bool issued = false;                                      // products issued (warp 8)

  // Registers: 384 x 168 at launch = 256 x 208 + 128 x 88.  A softmax thread holds a row of S.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ softmax of tile t, row r
    const int t = warp >> 2, r = threadIdx.x & 127;
    const int tok = tok0 + t * tq + r / p.pack, head = h0 + r % p.pack;
    const int lim = min(shift + tok, kv_len - 1);                     // last attended position
    const int sure = shift + tok0 + t * tq;                           // attended by every row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lanes + t * 128, to = tbase + lanes + 256 + t * HD;
    const int nt = n_t[t];
    float m = -INFINITY, l = 0.0f;  // m: the base of the exponents
    bool good = true;
    for (int j = 0; j < nt; ++j) {
      if (!(good = __all_sync(0xffffffffu, mbar_wait(&s_full[t], j & 1, abort_p, kPWait)))) break;
      tc_fence_after();
      float x[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, reinterpret_cast<uint32_t*>(x) + c * 32);
      tmem_ld_wait();
      if (j * kTile + kTile - 1 > sure) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (j * kTile + c > lim) x[c] = -INFINITY;
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c < 128; ++c) asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx[c & 3]) : "f"(x[c]));
      float top = mx[0];
#pragma unroll
      for (int c = 1; c < 4; ++c) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(mx[c]));
      const bool grown = !((top - m) * p.scale2 <= kGrow);  // not comparable: a NaN, or nothing attended yet
      if (__any_sync(0xffffffffu, grown)) {
        float f = 1.0f;  // a row's result does not depend on the rows beside it
        if (grown) {
          const float was = m;
          asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(top));
          f = was == -INFINITY ? 0.0f : ex2((was - m) * p.scale2);
          l *= f;
        }
        if (j > 0) {
          if (!(good = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (j - 1) & 1, abort_p, kPWait)))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < HD; c += 16) {
            uint32_t o[16];
            tmem_ld16(to + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(to + c, o);
          }
        }
      }
      const float neg = m == -INFINITY ? 0.0f : -m * p.scale2;  // nothing attended yet
      const uint64_t neg2 = pair(neg, neg), scale2 = pair(p.scale2, p.scale2);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 e = unpair(fma2(pair(x[c + 2 * i], x[c + 2 * i + 1]), scale2, neg2));
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          sum[i & 1] = add2(sum[i & 1], pair(e.x, e.y));
          w[i] = pack16<BF16>(e.x, e.y);
        }
        tmem_st16(ts + c / 2, w);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[t]);
      const float2 total = unpair(add2(sum[0], sum[1]));
      l += total.x + total.y;
    }
    if (good && nt > 0) {
      good = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (nt - 1) & 1, abort_p, kPWait));
      tc_fence_after();
    }
    if (good && tok0 + t * tq < n_q) {
      const bool attends = nt > 0 && lim >= 0 && m != -INFINITY;
      const float inv = 1.0f / l;
      const bool store = tok < n_q;
      uint16_t* out = p.out + ((size_t)(job.q0 + tok) * p.n_heads + head) * HD;
      const bool fix = *(volatile int*)&dirty != 0;
#pragma unroll
      for (int c = 0; c < HD; c += 16) {
        uint32_t o[16];
        if (nt > 0) {  // warp-uniform
          tmem_ld16(to + c, o);
          tmem_ld_wait();
        }
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = attends ? __uint_as_float(o[i]) * inv : 0.0f;
        if (fix && store) {
          // the values that were taken out of V, for the positions that this row attends
          for (int pos = max(0, shift + tok0 + 1); pos <= lim; ++pos) {
            const uint16_t* src = p.v + ((size_t)row[pos / s.page] * s.kv + kvh) * s.block_elems() + (size_t)(pos % s.page) * HD + c;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float v = unpack16<BF16>(src[i]);
              if (!isfinite(v)) y[i] += v;
            }
          }
        }
        if (store) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack16<BF16>(y[2 * i], y[2 * i + 1]);
          *reinterpret_cast<uint4*>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    }
    tc_fence_before();
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 8) {
    // ------------------------------------------------------------ products
    bool good = n > 0 && mbar_wait(&q_full, 0, abort_p, kPWait);
    good = __all_sync(0xffffffffu, good);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (good) good = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_p, kPWait));
      return good;
    };
    const uint64_t q_desc[2] = {sdesc_sw128(smem_addr(qs), 16, 1024), sdesc_sw128(smem_addr(qs + kOperand), 16, 1024)};
    auto scores = [&](int t, int j) {  // S_t = Q_t K(j)^T
      const int i = 2 * j;
      const uint64_t b = sdesc_sw128(smem_addr(ring + (i % kSlots) * kOperand), 16, 1024);
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        const uint64_t off = (uint64_t)(((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4);
        mma_ss(tbase + t * 128, q_desc[t] + off, b + off, kIdS, k != 0);
      }
      mma_commit(&s_full[t]);
      if (t == 1 || j >= n_t[1]) mma_commit(&empty[i % kSlots]);
    };
    auto product = [&](int t, int j) {  // O_t += P_t V(j)
      const int i = 2 * j + 1;
      const uint64_t b = sdesc_sw128(smem_addr(ring + (i % kSlots) * kOperand), kTile * 128, 1024);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts(tbase + 256 + t * HD, tbase + t * 128 + k * 8, b + (uint64_t)((k * 2048) >> 4), kIdO, (j | k) != 0);
      mma_commit(&o_done[t]);
      if (t == 1 || j >= n_t[1]) mma_commit(&empty[i % kSlots]);
    };
    if (good && wait(&full[0], 0)) {
      tc_fence_after();
      if (elect_one()) {
        if (n_t[0] > 0) scores(0, 0);
        if (n_t[1] > 0) scores(1, 0);
      }
      __syncwarp();
      issued = true;
    }
    for (int j = 0; j < n && good; ++j) {
      const int i = 2 * j + 1;
      if (!wait(&full[i % kSlots], (i / kSlots) & 1)) break;
      if (j == dirty_from - 1 && lane == 0) mbar_arrive(&near);
      if (j >= dirty_from && !wait(&clean[j % kVSlots], ((j - dirty_from) / kVSlots) & 1)) break;
      if (j + 1 < n && !wait(&full[(i + 1) % kSlots], ((i + 1) / kSlots) & 1)) break;
      for (int t = 0; t < 2; ++t) {
        if (j >= n_t[t]) continue;
        if (!wait(&p_full[t], j & 1)) break;
        tc_fence_after();
        if (elect_one()) {
          product(t, j);
          if (j + 1 < n_t[t]) scores(t, j + 1);
        }
        __syncwarp();
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ loads
    const int per = kTile / s.page;  // pages of a tile
    if (n > 0) {
      if (lane == 0) {
        mbar_expect_tx(&q_full, 2 * kOperand);
        for (int t = 0; t < 2; ++t)
          for (int h = 0; h < HD / 64; ++h)
            tma_load_3d(qs + t * kOperand + h * (kTile * 128), &tmQ, h * 64, h0, job.q0 + tok0 + t * tq, &q_full);
      }
      bool good = true;
      for (int j = 0; j < n && good; ++j) {
        const int pos = j * kTile + lane * s.page;
        const int pg = lane < per && pos < kv_len ? row[pos / s.page] : -1;
        const int held = __popc(__ballot_sync(0xffffffffu, pg >= 0));
        for (int kv = 0; kv < 2 && good; ++kv) {
          const int i = 2 * j + kv, slot = i % kSlots;
          if (i >= kSlots) good = __all_sync(0xffffffffu, mbar_wait(&empty[slot], (i / kSlots - 1) & 1, abort_p, kPWait));
          if (!good) break;
          if (lane == 0) mbar_expect_tx(&full[slot], held * s.page * HD * 2);
          __syncwarp();
          loads = i + 1;
          if (pg >= 0)
            for (int h = 0; h < HD / 64; ++h)
              tma_load_3d(ring + slot * kOperand + h * (kTile * 128) + lane * s.page * 128, kv ? &tmV : &tmK, h * 64, 0,
                          pg * s.kv + kvh, &full[slot]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ V tiles with positions not every row attends
    const int me = threadIdx.x - 320;
    constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
    // A full barrier's parity means something only to a waiter that knows the phase before has passed: for
    // the uses before the first dirty tile the product warp, which waits for each, says so.
    bool good = dirty_from == 0 || dirty_from >= n || mbar_wait(&near, 0, abort_p, kPWait);
    for (int j = dirty_from; j < n && good; ++j) {
      const int i = 2 * j + 1, slot = i % kSlots;
      if (!(good = mbar_wait(&full[slot], (i / kSlots) & 1, abort_p, kPWait))) break;
      uint8_t* tile = ring + slot * kOperand;
      for (int e = me; e < kTile * HD / 8; e += 64) {
        const int pos = j * kTile + ((e >> 3) & 127);
        uint4* at = reinterpret_cast<uint4*>(tile + e * 16);  // [half][row][8 chunks]; a row's chunks stay in it
        if (pos >= kv_len) {
          *at = make_uint4(0, 0, 0, 0);
        } else if (pos > shift + tok0) {
          uint4 x = *at;
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if ((w[k] & kExp) == kExp) bad = true, w[k] &= 0xffff0000u;
            if (((w[k] >> 16) & kExp) == kExp) bad = true, w[k] &= 0x0000ffffu;
          }
          if (bad) {
            *at = make_uint4(w[0], w[1], w[2], w[3]);
            *(volatile int*)&dirty = 1;
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&clean[j % kVSlots]);  // one barrier a slot: the cleaning may run ahead of the products
    }
  }
  }

  __syncthreads();
  if (abort_flag) {
    // an abandoned pipeline: neither may products still write TMEM when it is freed, nor loads shared
    // memory when the CTA exits (bounded waits)
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    const long long t0 = clock64();
    if (warp == 8 && issued) {
      if (elect_one()) mma_commit(&fin);
      __syncwarp();
      while (!mbar_try_wait(&fin, 0) && clock64() - t0 < kPWait) {
      }
    }
    if (warp == 9 && n > 0) {
      while (!mbar_try_wait(&q_full, 0) && clock64() - t0 < kPWait) {
      }
      for (int i = max(0, loads - kSlots); i < loads; ++i)
        while (!mbar_try_wait(&full[i % kSlots], (i / kSlots) & 1) && clock64() - t0 < kPWait) {
        }
    }
    __syncthreads();
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// 16-bit tensor map [z][y][x], row pitches in bytes, box [box_z][box_y][64], 128-byte swizzle.
bool make_tmap3(CUtensorMap* tm, const void* base, bool bf16, uint64_t x, uint64_t y, uint64_t z, uint64_t pitch_y,
                uint64_t pitch_z, uint32_t box_y, uint32_t box_z) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {x, y, z}, strides[2] = {pitch_y, pitch_z};
  const cuuint32_t box[3] = {64, box_y, box_z}, estr[3] = {1, 1, 1};
  return enc(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool BF16>
cudaError_t launch_as(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, const PromptParams& p,
                      cudaStream_t st) {
  int limit = 0;
  cudaError_t e = dyn_smem_limit((const void*)paged_prompt_kernel<HD, BF16>, &limit);
  if (e != cudaSuccess) return e;
  if (PromptSmem<HD>::kBytes > limit) return cudaErrorInvalidConfiguration;
  const int tq = kTile / p.pack;
  const long long blocks = (long long)p.n_rows / (2 * tq) + p.n_lanes;  // at least the lanes' blocks
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)(blocks * (p.n_heads / p.pack)));
  cfg.blockDim = dim3(kPromptThreads);
  cfg.dynamicSmemBytes = PromptSmem<HD>::kBytes;
  profile_stream_begin(st);
  e = cudaLaunchKernelEx(&cfg, paged_prompt_kernel<HD, BF16>, tmQ, tmK, tmV, p);
  profile_stream_end(st);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_prompt(const PagedPromptArgs& a, cudaStream_t st) {
  const PagedShape& s = a.s;
  const size_t off = (size_t)a.layer * s.layer_elems();
  const int group = a.n_heads / s.kv;
  int pack = group & -group;  // largest power of two that divides the group
  if (pack > kTile) pack = kTile;
  const bool bf16 = s.dtype == TL_KV_BF16;
  alignas(64) CUtensorMap tmQ, tmK, tmV;
  const uint64_t blocks = (uint64_t)s.n_pages * s.kv;
  if (!make_tmap3(&tmQ, a.q, bf16, s.hd, a.n_heads, a.n_rows, s.hd * 2, (uint64_t)a.q_stride * 2, pack, kTile / pack) ||
      !make_tmap3(&tmK, a.c.k + off, bf16, s.hd, s.page, blocks, s.hd * 2, s.block_elems() * 2, s.page, 1) ||
      !make_tmap3(&tmV, a.c.v + off, bf16, s.hd, s.page, blocks, s.hd * 2, s.block_elems() * 2, s.page, 1))
    return cudaErrorInvalidValue;
  const PromptParams p{s,      a.c.v + off, a.c.table,           a.cu_q,         a.kv_len, a.seqs,
                       (uint16_t*)a.out, (uint32_t*)a.ws, a.scale * kLog2e, a.n_heads, group, pack, a.n_rows, a.n_lanes};
  if (s.hd == 64) return bf16 ? launch_as<64, true>(tmQ, tmK, tmV, p, st) : launch_as<64, false>(tmQ, tmK, tmV, p, st);
  return bf16 ? launch_as<128, true>(tmQ, tmK, tmV, p, st) : launch_as<128, false>(tmQ, tmK, tmV, p, st);
}

}  // namespace tl
