// Causal attention of packed prompts over the paged K/V cache (tl_paged_prompt_attn) on
// 5th-generation tensor cores (tcgen05 + TMEM), sm_100a.
//
// Per (lane, query head): S = Q K^T, P = exp2((S - m) scale log2 e) with m the running row maximum,
// O = P V / rowsum(P), one pass over K and V.  4 x hd operations per attended pair: the tensor pipe
// bounds long prompts, and next to it the exponentials (16 a clock and SM: as many clocks as the two products
// at hd = 128).
//
// Work: a block is two tiles of 128 query rows.  A row is a (token, head) pair: the Gp heads of one
// K/V head that fit (Gp the largest power of two up to 128 dividing the group) lie next to each
// other, 128 / Gp tokens a tile, so the heads of a group share their K and V and the causal edge is
// only 128 / Gp tokens wide.  Persistent CTAs, one per SM, take blocks from a counter, a lane's last
// and longest first; blocks beyond the last full round over the SMs are cut along their positions into
// pieces whose (maximum, sum, O) are joined, in the order of the pieces, by the last one to finish.
//
// Positions come in steps of 64.  Roles of a CTA's warps:
//   0-3, 4-7  softmax of tile 0 / 1, a thread per row: S from TMEM, maximum, P back over S's columns
//             as 16-bit values (A operand of the second product), at the end O / sum
//   8, 11     issue the products of tile 0 / 1 (a warp each: the waits of one, some 100 clocks even
//             when there is nothing to wait for, pass behind the products of the other).  Each tile has
//             two S buffers of 64 columns: S_t(u+2) is issued behind P_t(u) V(u), so that the next S
//             is there while a tile's softmax runs and the tensor pipe has products meanwhile
//   9, 10     load by TMA, page by page (a page of one K/V head is one box per 64 values): Q and K / V.  A slot of the ring holds what one issue of products takes, K(u+2) and V(u).
//             (Two warps: a box costs some 50 clocks of issue, a step of 16-position pages 16 boxes.)
//             Warp 9 also cleans, with 13 to 15, the V steps that hold positions not every row attends: rows
//             past the cache's end are zeroed (their memory may hold anything) and values that are not finite are
//             taken out (0 x inf would reach the rows that do not attend them) and given back at the end
//             to the rows that do
//   12        takes work (a job: a block or a piece of one) and looks its lane's pages over, 3 us ahead
// O is rescaled only when a row's maximum has grown by more than 2^8 in the exponent since the last
// time: the base of the exponents is a free choice (P then reaches 2^8, in FP16 2^15, and its sum that times the
// positions, far inside FP32), and the rescale, a round trip of O through registers, becomes rare.
//
// Precision: scores, statistics, sums and O in FP32.  P is rounded to the cache's type for the second product: half a
// step, 2^-8 (BF16) or 2^-11 (FP16) relative, and in FP16 at least 2^-32 of the row's base; the sum is of the unrounded
// P.  (60000 FP16 positions 17.6 natural units below the first one keep their 0.14% of the weight.)
//
// Measured: 16384 tokens, 16 heads over 4 K/V heads x 128, 915 to 940 us in long loops (1.17 to 1.20 PFLOP/s, power
// bound: the clock falls to 1.40 GHz), 820 us in short ones at 1.59 GHz: about 1380 clocks a step, the two tiles'
// products being 1024 at the tensor pipe's rate, or 1280 with the scores' operands (6 KB a product of 128 x 64 x 16)
// at 128 bytes a clock from shared memory; the exponentials 1024.  Steps of 128 with one S buffer a tile took 1720
// (softmax, then products, one behind the other); the exponentials of the two tiles taking turns on a scheduler,
// 1600.  A job costs about 6000 clocks besides its steps: 1100 until its last product is done, 2400 for O / sum and its
// stores, 1200 for the next one's first softmax; a CTA's first job starts 11 000 clocks after the launch, by the chain
// of loads of the work, the pages, Q and K and by code that is fetched for the first time.
//
// TMEM (512 columns): S_0 (two buffers) | S_1 (128 columns each; P over a buffer's first 32) | O_0 | O_1.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <mutex>

#include "paged_internal.cuh"
#include "tc_ptx.cuh"

namespace tl {
namespace {

using namespace ptx;

constexpr int kPromptThreads = 512;
constexpr int kTile = 128;                // query rows of a tile
constexpr int kStep = 64;                 // positions of a step
constexpr int kSms = 148;
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;  // of 128 at launch
constexpr int kAhead = 8;                 // turns before a job's last that the next one is taken
constexpr long long kPWait = 4000000000ll;  // SM clocks
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;  // growth of the maximum, in powers of two, that O is rescaled for
// FP16's exponents end soon: P is held 2^7 times as large, at most 2^15 then (of 65504), and the weights that FP16 spaces
// 2^-24 apart are those below 2^-21 of the row's base instead of 2^-14.  Sums and O carry the factor alike.  BF16 has
// FP32's exponents and needs none.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;

// ptx::mbar_wait for the many waits of this kernel, whose code shares the instruction caches with the softmax's:
// tries in one place, and for the roles that are not softmax (whose registers leave no room for a call) with what
// comes behind the first look in a function.  Measured, with the loops over O's rescale and a V step's cleaning rolled
// up as well: packed prompts 192 -> 185 us a call, 130 tokens 11.0 -> 10.4, chunks 213 -> 209.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
  long long t0 = 0;
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    const long long t = clock64();
    if (t0 == 0) t0 = t;
    if (t - t0 > kPWait) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort) { return wait_for(bar, parity, abort); }
__device__ __forceinline__ bool wait_apart(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort);
}

// For a wait that may span any number of jobs: the limit starts anew with each job that the CTA takes.
__device__ __noinline__ bool wait_over_jobs(uint64_t* bar, uint32_t parity, volatile int* abort, volatile const int* taken) {
  int seen = *taken;
  long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    const int now = *taken;
    const long long t = clock64();
    if (now != seen) {
      seen = now;
      t0 = t;
    }
    if (t - t0 > kPWait) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

struct PromptParams {
  PagedShape s;
  const uint16_t* v;  // the layer's
  const int32_t* table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* seqs;
  uint16_t* out;
  uint32_t* status;
  int32_t* queue;     // [0]: blocks taken beyond the first of each CTA, [1]: CTAs done; both 0 between calls
  int32_t* finished;  // [kPromptPieces][2] pieces of a block that are done, per tile; 0 between calls
  float* part;        // [kPromptPieces][2] x (maximum and sum [128][2] | O [HD][128])
  float scale2;       // scale * log2 e
  int n_heads, group, pack, n_rows, n_lanes, pieces;
};

template <int HD>
struct PromptSmem {
  static constexpr int kQ = kTile * HD * 2;     // one tile of queries
  static constexpr int kKv = kStep * HD * 2;    // one step of K or of V
  static constexpr int kSlots = 4;              // of each ring
  static constexpr int kStage = 8 * 2 * 32 * 64;  // of the outputs, a softmax warp's rows x 32 values, twice
  static constexpr int kBytes = 1024 + 2 * kQ + 2 * kSlots * kKv + kStage;
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
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

// x, the same for every lane of the warp, in a form that the compiler knows to be: what the products are issued with
// then lies in uniform registers.
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// What a CTA works on.
struct Job {
  int lane;     // -1: no more
  int q0, n_q;  // first packed row and number of queries of the lane
  int kv, seq;  // cached positions, sequence
  int tok0;     // first token of the first tile
  int head0, kvh;
  int u0, n;    // first step of the piece, steps
  int n_t[2];   // of them, those that tile t attends
  int dirty_from;  // first step of the piece with positions that not every row attends
  int slot, piece, pieces;  // where partial results go: (block, heads) and piece
  int dirty;    // a value that is not finite was taken out of V
};

// A V step to clean: its slot (-1: no more), the first row that not every query row attends, the first row past
// the cache's end, and where to note that a value was taken out.
struct Dirty {
  int slot, row, end;
  int* noted;
};
// Share `part` of four of it, by one warp: 4 rows in 16.
template <int HD, bool BF16>
__device__ __forceinline__ void clean_step(uint8_t* tile, const Dirty& d, int part) {
  constexpr uint32_t kExp = BF16 ? 0x7f807f80u : 0x7c007c00u, kOne = BF16 ? 0x00800080u : 0x04000400u;
  const int lane = threadIdx.x & 31;
  bool found = false;
#pragma unroll 1
  for (int r = d.row + part * 4 + (lane >> 3); r < kStep; r += 16) {
#pragma unroll
    for (int h = 0; h < HD / 64; ++h) {
      uint4* at = reinterpret_cast<uint4*>(tile + h * (kStep * 128) + r * 128 + (lane & 7) * 16);
      uint4 x = *at;
      // a sign bit for every exponent that is all ones
      const uint32_t bad = (((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne)) & 0x80008000u;
      if (r >= d.end) {
        *at = make_uint4(0, 0, 0, 0);
      } else if (bad) {
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t b = (w[k] & kExp) + kOne;
          w[k] &= (b & 0x8000u ? 0u : 0xffffu) | (b & 0x80000000u ? 0u : 0xffff0000u);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
        found = true;
      }
    }
  }
  if (found) *(volatile int*)d.noted = 1;
  fence_proxy_async_smem();
}

// What the warps of a tile agree on when its block is cut into pieces.
struct Joint {
  uint64_t done[2], said[2];  // the piece's part is written; whether it is the last one is known
  int last[2];
};

// 32 values of every row of a warp into shared memory (64-byte rows, 64-byte swizzle), in two buffers by turns.  Every
// use of a buffer commits one bulk group, an empty one where no TMA store reads it, so that "all groups but the newest"
// are those of this buffer's last use and before.
__device__ __forceinline__ uint32_t stage_words(uint32_t stage, int d, const uint32_t* w) {
  const int lane = threadIdx.x & 31;
  const uint32_t buf = stage + (d / 32 & 1) * 2048;
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the store before the last has read this buffer
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)),
                 "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                 : "memory");
  return buf;
}
// From there into the output: by one TMA store, where all rows are the lane's.
__device__ __forceinline__ void store_rows(const CUtensorMap* tmO, int d, int head, int row, uint32_t buf) {
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(tmO)),
                 "r"(d), "r"(head), "r"(row), "r"(buf)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// Where some are not: four lanes write 64 bytes of a row.  The empty group keeps the count of stage_words: without it
// the one group left pending could be a store of the job before that still reads the buffer written next.
template <int HD>
__device__ __forceinline__ void copy_rows(const PromptParams& p, const Job& job, int first, int log_pack, int row0, int d,
                                          uint32_t buf) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int wr = i * 8 + (lane >> 2), row = row0 + wr, to_tok = first + (row >> log_pack);
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(buf + wr * 64 + (((lane & 3) ^ ((wr >> 1) & 3)) << 4))
                 : "memory");
    if (to_tok < job.n_q)
      *reinterpret_cast<uint4*>(p.out + ((size_t)(job.q0 + to_tok) * p.n_heads + job.head0 + (row & ((1 << log_pack) - 1))) * HD + d +
                                (lane & 3) * 8) = v;
  }
  if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The end of a tile's job where the usual one does not do: a tile that attends nothing; values to give back; the part of
// a piece into the workspace and, by the last piece, the parts joined.  False: a wait gave up.
template <int HD, bool BF16>
__device__ __noinline__ bool finish_rare(const PromptParams& p, const CUtensorMap* tmO, const Job& job, int t,
                                         int log_pack, uint32_t to, uint32_t stage, float m, float l, Joint* joint,
                                         int& parts, volatile int* abort) {
  constexpr int kPartFloats = kTile * (HD + 2);
  const PagedShape& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x & 127;
  const int tq = kTile >> log_pack, first = job.tok0 + t * tq, shift = job.kv - job.n_q;
  const int tok = first + (r >> log_pack), lim = min(shift + tok, job.kv - 1);
  const int nt = job.n_t[t], pos0 = job.u0 * kStep;
  bool good = true;
  const bool attends = nt > 0 && lim >= 0 && m != -INFINITY;
  const bool store = tok < job.n_q;
  const int fix0 = max(max(0, shift + job.tok0 + 1), pos0), fix1 = min(lim, pos0 + job.n * kStep - 1);
  const bool fix = *(volatile const int*)&job.dirty != 0 && store;
  const int32_t* row = p.table + (size_t)job.seq * s.max_pages;
  // the values that were taken out of V, for the positions that this row attends
  auto give_back = [&](int d, float* y) {
    for (int pos = fix0; pos <= fix1; ++pos) {
      const uint16_t* src = p.v + ((size_t)row[pos / s.page] * s.kv + job.kvh) * s.block_elems() + (size_t)(pos % s.page) * HD + d;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float v = unpack16<BF16>(src[i]);
        if (!isfinite(v)) y[i] += v;
      }
    }
  };
  const int row0 = (warp & 3) * 32;
  const bool all = first + ((row0 + 31) >> log_pack) < job.n_q;
  const int to_head = job.head0 + (row0 & ((1 << log_pack) - 1)), to_row = job.q0 + first + (row0 >> log_pack);
  auto put = [&](int d, const float* y) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack16<BF16>(y[2 * i], y[2 * i + 1]);
    const uint32_t buf = stage_words(stage, d, w);
    if (all) {
      store_rows(tmO, d, to_head, to_row, buf);
      return;
    }
    copy_rows<HD>(p, job, first, log_pack, row0, d, buf);
  };
  if (job.pieces == 1) {
    const float inv = 1.0f / l;
#pragma unroll 1
    for (int d = 0; d < HD; d += 32) {
      uint32_t o[32];
      if (nt > 0) {  // warp-uniform
        tmem_ld32(to + d, o);
        tmem_ld_wait();
      }
      float y[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        asm volatile("" : "+r"(o[i]));
        y[i] = attends ? __uint_as_float(o[i]) * inv : 0.0f;
      }
      if (fix) give_back(d, y);
      put(d, y);
    }
  } else {
    // leave the piece's part; the last piece of the tile to come by joins them all in their order
    float* part = p.part + ((size_t)(job.slot + job.piece) * 2 + t) * kPartFloats;
    reinterpret_cast<float2*>(part)[r] = make_float2(attends ? m : -INFINITY, l);
    if (nt > 0) {
#pragma unroll 1
      for (int d = 0; d < HD; d += 32) {
        uint32_t o[32];
        tmem_ld32(to + d, o);
        tmem_ld_wait();
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          asm volatile("" : "+r"(o[i]));
          y[i] = __uint_as_float(o[i]);
        }
        if (fix) give_back(d, y);
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          reinterpret_cast<float4*>(part + 2 * kTile)[(d + i) / 4 * kTile + r] = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
      }
    }
    __threadfence();
    mbar_arrive(&joint->done[t]);
    if (r == 0 && (good = wait_for(&joint->done[t], parts & 1, abort))) {
      __threadfence();
      int32_t* count = p.finished + job.slot * 2 + t;
      const bool last = atomicAdd(count, 1) == job.pieces - 1;
      if (last) *count = 0;
      joint->last[t] = last;
      mbar_arrive(&joint->said[t]);
    }
    good = __all_sync(0xffffffffu, good && wait_for(&joint->said[t], parts & 1, abort));
    if (!good) return false;
    ++parts;
    if (*(volatile int*)&joint->last[t]) {
      __threadfence();
      const float* base = p.part + ((size_t)job.slot * 2 + t) * kPartFloats;
      const size_t next = 2 * kPartFloats;  // the following piece's
      float f[kPromptMostPieces], top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kPromptMostPieces; ++i) {
        f[i] = i < job.pieces ? __ldcg(base + i * next + 2 * r) : -INFINITY;
        top = fmaxf(top, f[i]);
      }
#pragma unroll
      for (int i = 0; i < kPromptMostPieces; ++i) {
        // a NaN stays one; a piece of which the row attends nothing counts for nothing
        f[i] = f[i] == -INFINITY ? 0.0f : ex2((f[i] - top) * p.scale2);
        if (f[i] != 0.0f) sum = fmaf(__ldcg(base + i * next + 2 * r + 1), f[i], sum);
      }
      const float inv = top == -INFINITY ? 0.0f : 1.0f / sum;
#pragma unroll 1
      for (int d = 0; d < HD; d += 32) {
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < kPromptMostPieces; ++k)
          if (f[k] != 0.0f) {
            float4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              x[i] = __ldcg(reinterpret_cast<const float4*>(base + k * next + 2 * kTile) + (d / 4 + i) * kTile + r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              y[4 * i] = fmaf(x[i].x, f[k], y[4 * i]);
              y[4 * i + 1] = fmaf(x[i].y, f[k], y[4 * i + 1]);
              y[4 * i + 2] = fmaf(x[i].z, f[k], y[4 * i + 2]);
              y[4 * i + 3] = fmaf(x[i].w, f[k], y[4 * i + 3]);
            }
          }
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] *= inv;
        put(d, y);
      }
    }
  }
  return true;
}

// The end of a tile's job, by the threads of its rows: O / l into the output.  The cases that are rare or long are a
// function apart, which the main loop is the faster for (packed prompts 187 -> 184 us a call, chunks 214 -> 211); with
// this loop unrolled the larger code cost more than it saved (packed prompts 214, 16384 tokens 962 against 925).
template <int HD, bool BF16>
__device__ __forceinline__ bool finish_rows(const PromptParams& p, const CUtensorMap* tmO, const Job& job, int t,
                                            int log_pack, uint32_t to, uint32_t stage, float m, float l, Joint* joint,
                                            int& parts, volatile int* abort) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x & 127;
  const int tq = kTile >> log_pack, first = job.tok0 + t * tq, nt = job.n_t[t], row0 = (warp & 3) * 32;
  const bool all = first + ((row0 + 31) >> log_pack) < job.n_q;
  if (first >= job.n_q) return true;  // a tile without tokens
  // one answer for the warp: a step that only the other tile attends may be under cleaning still
  if (job.pieces > 1 || nt == 0 || __any_sync(0xffffffffu, *(volatile const int*)&job.dirty != 0))
    return finish_rare<HD, BF16>(p, tmO, job, t, log_pack, to, stage, m, l, joint, parts, abort);
  const int to_head = job.head0 + (row0 & ((1 << log_pack) - 1)), to_row = job.q0 + first + (row0 >> log_pack);
  const int lim = min(job.kv - job.n_q + first + (r >> log_pack), job.kv - 1);
  const bool attends = lim >= 0 && m != -INFINITY;
  const float inv = 1.0f / l;
  const uint64_t inv2 = pair(inv, inv);
#pragma unroll 1
  for (int d = 0; d < HD; d += 32) {
    uint32_t o[32], w[16];
    tmem_ld32(to + d, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(o[i]));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 y = unpair(mul2(pair(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), inv2));
      w[i] = attends ? pack16<BF16>(y.x, y.y) : 0u;
    }
    const uint32_t buf = stage_words(stage, d, w);
    if (all)
      store_rows(tmO, d, to_head, to_row, buf);
    else
      copy_rows<HD>(p, job, first, log_pack, row0, d, buf);
  }
  return true;
}

template <int HD, bool BF16>
__global__ void __launch_bounds__(kPromptThreads, 1)
    paged_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                        const __grid_constant__ PromptParams p) {
  using Smem = PromptSmem<HD>;
  constexpr int kSlots = Smem::kSlots;
  constexpr uint32_t kIdS = idesc16<BF16>(128, kStep, false), kIdO = idesc16<BF16>(128, HD, true);
  extern __shared__ uint8_t smem_raw[];
  // A wait by parity cannot tell a phase from the second one behind it, so every barrier is waited for in
  // each of its phases in turn, or its next phase needs the waiter; what may be two steps behind has two.
  __shared__ uint64_t q_full, q_empty, full[kSlots], empty[kSlots], clean[kSlots];
  __shared__ uint64_t s_full[2][2], p_full[2][2], o_done[2][2], job_full[2], job_empty[2], fin[2];
  __shared__ uint32_t tmem_base;
  __shared__ uint64_t want, go;
  __shared__ Dirty dirt;
  __shared__ int abort_flag, jobs_taken;
  __shared__ Joint joint_mem;
  Joint* joint = &joint_mem;
  __shared__ Job jobs[2];
  uint8_t* qs = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);  // two tiles
  uint8_t* ks = qs + 2 * Smem::kQ;
  uint8_t* vs = ks + kSlots * Smem::kKv;

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  const PagedShape& s = p.s;
  const int subs = p.n_heads / p.pack, tq = kTile / p.pack;
  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&want, 1);
    mbar_init(&go, 1);
    mbar_init(&q_empty, 2);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 2);   // K's and V's loads
      mbar_init(&empty[i], 2);  // both tiles
      mbar_init(&clean[i], 128);  // four warps
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[t][i], 1);
        mbar_init(&p_full[t][i], 128);
        mbar_init(&o_done[t][i], 1);
      }
      mbar_init(&fin[t], 1);
      mbar_init(&joint->done[t], 128);
      mbar_init(&joint->said[t], 1);
      mbar_init(&job_full[t], 1);
      mbar_init(&job_empty[t], 12);  // warps that read a job
    }
    abort_flag = 0;
    jobs_taken = 0;
    mbar_fence_init();
  }
  pdl_wait();
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
  bool issued = false;                 // products issued (warps 8, 11)
  int q_loads = 0, loads = 0;          // jobs and slots loaded (warps 9, 10)

  // Loads a job's steps of K (behind 0) or V (behind 2) into ring: step u into slot loads + u + behind.
  const int box = min(s.page, kStep), per = kStep / box;  // rows of a TMA box, boxes of a step
  const int wide = s.page / box - 1;                      // 1: a page is two boxes (128 positions)
  auto load_steps = [&](const Job& job, const CUtensorMap* tm, uint8_t* ring, int behind, auto before) {
    const int32_t* row = p.table + (size_t)job.seq * s.max_pages;
    // pages of 32 boxes at a time, one per lane, and of the 32 behind them
    auto pages_at = [&](int i) {
      const int e = job.u0 * per + i + lane;
      return e * box < job.kv && i < job.n * per ? row[e >> wide] : 0;
    };
    int pages = pages_at(0), pages_next = pages_at(32);
    for (int w = 0; w < job.n + 2; ++w, ++loads) {
      const int slot = loads % kSlots, u = w - behind, pos = (job.u0 + u) * kStep;
      if (!before(w)) return false;
      if (loads >= kSlots && !__all_sync(0xffffffffu, wait_for(&empty[slot], (loads / kSlots - 1) & 1, abort_p))) return false;
      if (u < 0 || u >= job.n) {
        if (lane == 0) mbar_arrive(&full[slot]);
        continue;
      }
      const int at = u * per & 31;
      if (at == 0 && u > 0) {
        pages = pages_next;
        pages_next = pages_at(u * per + 32);
      }
      const int page = __shfl_sync(0xffffffffu, pages, (at + lane) & 31);
      const int boxes = min(per, (job.kv - pos + box - 1) / box);
      if (lane == 0) mbar_expect_tx(&full[slot], boxes * box * HD * 2);
      if (lane < boxes) {
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
          tma_load_3d(ring + slot * Smem::kKv + h * (kStep * 128) + lane * box * 128, tm, h * 64, pos & (s.page - 1),
                      page * s.kv + job.kvh, &full[slot]);
      }
      __syncwarp();
    }
    return true;
  };

  // Registers: 512 x 128 at launch = 256 x 184 (softmax: a thread holds a row of S) + 256 x 72.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax of tile t, row r
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lanes + t * 128, to = tbase + lanes + 256 + t * HD;
    const uint32_t stage = smem_addr(vs + kSlots * Smem::kKv) + warp * 4096;  // twice 32 rows x 64 bytes
    const int log_pack = __ffs(p.pack) - 1;
    int c = 0, parts = 0;  // steps of this tile and partial results so far
    bool good = true;
    for (int nj = 0; good; ++nj) {
      if (!(good = __all_sync(0xffffffffu, wait_for(&job_full[nj & 1], (nj >> 1) & 1, abort_p)))) break;
      const Job& job = jobs[nj & 1];
      if (job.lane < 0) break;
      const int first = job.tok0 + t * tq, shift = job.kv - job.n_q;  // shift: position of token 0
      const int tok = first + (r >> log_pack);
      const int lim = min(shift + tok, job.kv - 1);  // last attended position
      const int sure = shift + first;                // attended by every row of the tile
      const int nt = job.n_t[t], pos0 = job.u0 * kStep;
      float m = -INFINITY, l = 0.0f;  // m: the base of the exponents
      for (int u = 0; u < nt; ++u, ++c) {
        const int buf = c & 1;
        if (!(good = __all_sync(0xffffffffu, wait_for(&s_full[t][buf], (c >> 1) & 1, abort_p)))) break;
        tc_fence_after();
        float x[kStep];
        tmem_ld32(ts + buf * kStep, reinterpret_cast<uint32_t*>(x));
        tmem_ld32(ts + buf * kStep + 32, reinterpret_cast<uint32_t*>(x) + 32);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < kStep; ++i) asm volatile("" : "+f"(x[i]));  // nothing of x is used before the wait
        const int pos = pos0 + u * kStep;
        if (pos + kStep - 1 > sure) {
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            if (pos + i > lim) x[i] = -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < kStep; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx[i & 3]) : "f"(x[i]));
        float top = mx[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(mx[i]));
        const bool grown = !((top - m) * p.scale2 <= kGrow);  // not comparable: a NaN, or nothing attended yet
        if (__any_sync(0xffffffffu, grown)) {
          float f = 1.0f;  // a row's result does not depend on the rows beside it
          if (grown) {
            const float was = m;
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(top));
            f = was == -INFINITY ? 0.0f : ex2((was - m) * p.scale2);
            l *= f;
          }
          if (u > 0) {
            if (!(good = __all_sync(0xffffffffu, wait_for(&o_done[t][(c - 1) & 1], ((c - 1) >> 1) & 1, abort_p)))) break;
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < HD; d += 16) {
              uint32_t o[16];
              tmem_ld16(to + d, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(to + d, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.0f : fmaf(-m, p.scale2, kLift<BF16>);  // nothing attended yet
        const uint64_t neg2 = pair(neg, neg), scale2 = pair(p.scale2, p.scale2);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int d = 0; d < kStep; d += 32) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 e = unpair(fma2(pair(x[d + 2 * i], x[d + 2 * i + 1]), scale2, neg2));
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[i & 1] = add2(sum[i & 1], pair(e.x, e.y));
            w[i] = pack16<BF16>(e.x, e.y);
          }
          tmem_st16(ts + buf * kStep + d / 2, w);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[t][buf]);
        const float2 total = unpair(add2(sum[0], sum[1]));
        l += total.x + total.y;
      }
      if (good && nt > 0) {
        good = __all_sync(0xffffffffu, wait_for(&o_done[t][(c - 1) & 1], ((c - 1) >> 1) & 1, abort_p));
        tc_fence_after();
      }
      if (!good) break;
      if (!(good = finish_rows<HD, BF16>(p, &tmO, job, t, log_pack, to, stage, m, l, joint, parts, abort_p))) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&job_empty[nj & 1]);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the outputs are written
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8 || warp == 11) {
      // ------------------------------------------------------------ products of tile t
      const int t = uniform(warp == 11);
      const uint32_t tbase = uniform(tmem_base);
      bool good = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (good) good = __all_sync(0xffffffffu, wait_apart(bar, parity, abort_p));
        return good;
      };
      const uint64_t q_desc = sdesc_sw128(smem_addr(qs + t * Smem::kQ), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_addr(ks), 16, 1024), v_desc = sdesc_sw128(smem_addr(vs), kStep * 128, 1024);
      const uint32_t ts = tbase + t * 128, to = tbase + 256 + t * HD;
      int at = 0, c = 0;         // slots, and steps of this tile, before this job
      uint32_t clean_phase = 0;  // one bit per slot
      for (int nj = 0; good; ++nj) {
        if (!wait(&job_full[nj & 1], (nj >> 1) & 1)) break;
        const Job& job = jobs[nj & 1];
        if (job.lane < 0) break;
        const int n = uniform(job.n), nt = uniform(job.n_t[t]), dirty_from = uniform(job.dirty_from);
        __syncwarp();
        if (lane == 0) mbar_arrive(&job_empty[nj & 1]);
        if (n == 0) continue;
        if (!wait(&q_full, nj & 1)) break;
        // turn w: O_t += P_t(w - 2) V(w - 2), then S_t(w) = Q_t K(w)^T; both operands lie in slot at + w
        for (int w = 0; w < n + 2; ++w) {
          const int slot = (at + w) % kSlots, u = w - 2;
          if (!wait(&full[slot], ((at + w) / kSlots) & 1)) break;
          if (u >= dirty_from && u >= 0) {
            if (!wait(&clean[slot], (clean_phase >> slot) & 1)) break;
            clean_phase ^= 1u << slot;
          }
          const bool pv = u >= 0 && u < nt, qk = w < nt;
          const int buf = (c + w) & 1;  // of step w and of step u
          if (pv && !wait(&p_full[t][buf], ((c + u) >> 1) & 1)) break;
          tc_fence_after();
          if (elect_one()) {
            if (pv) {
              const uint64_t b = v_desc + (uint64_t)((slot * Smem::kKv) >> 4);
#pragma unroll
              for (int k = 0; k < kStep / 16; ++k)
                mma_ts(to, ts + buf * kStep + k * 8, b + (uint64_t)((k * 2048) >> 4), kIdO, (u | k) != 0);
              mma_commit(&o_done[t][buf]);
            }
            if (qk) {
              const uint64_t b = k_desc + (uint64_t)((slot * Smem::kKv) >> 4);
#pragma unroll
              for (int k = 0; k < HD / 16; ++k)
                mma_ss(ts + buf * kStep, q_desc + (uint64_t)(((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4),
                       b + (uint64_t)(((k / 4) * (kStep * 128) + (k % 4) * 32) >> 4), kIdS, k != 0);
              mma_commit(&s_full[t][buf]);
            }
            // the slot is free once these products are done (at once where this tile attends neither), the queries
            // once all of this tile's scores are
            if (pv || qk)
              mma_commit(&empty[slot]);
            else
              mbar_arrive(&empty[slot]);
            if (w == n - 1) mma_commit(&q_empty);  // also where this turn has no scores: the last ones may still run
          }
          __syncwarp();
          issued = true;
        }
        at += n + 2;
        c += nt;
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ loads of Q and K
      // Has the next V steps of a job cleaned that need it, up to step `end`; `first` is the job's first slot.  (This
      // warp waited for the slots to be free, so it knows which phase of their loads it waits for.)  Four warps
      // share a step; the one before is done when the next is given out.
      int dirty_next = 0, last = -1;  // the slot given out last
      uint32_t clean_phase = 0;       // one bit per slot
      auto give_out = [&](const Dirty& d) {
        if (last >= 0) {
          if (!__all_sync(0xffffffffu, wait_apart(&clean[last], (clean_phase >> last) & 1, abort_p))) return false;
          clean_phase ^= 1u << last;
        }
        last = d.slot;
        if (lane == 0) {
          dirt = d;
          mbar_arrive(&go);
        }
        return true;
      };
      auto clean_steps = [&](Job& job, int first, int end) {
        for (; dirty_next < end; ++dirty_next) {
          const int i = first + dirty_next + 2, slot = i % kSlots, pos = (job.u0 + dirty_next) * kStep;
          if (!__all_sync(0xffffffffu, wait_apart(&full[slot], (i / kSlots) & 1, abort_p))) return false;
          // not attended by every row: the positions behind the first query's
          const Dirty d{slot, max(0, job.kv - job.n_q + job.tok0 + 1 - pos), job.kv - pos, &job.dirty};
          if (!give_out(d)) return false;
          clean_step<HD, BF16>(vs + slot * Smem::kKv, d, 0);
          mbar_arrive(&clean[slot]);
        }
        return true;
      };
      bool good = true;
      for (int nj = 0; good; ++nj) {
        if (!(good = __all_sync(0xffffffffu, wait_apart(&job_full[nj & 1], (nj >> 1) & 1, abort_p)))) break;
        const Job job = jobs[nj & 1];
        if (job.lane < 0) break;
        const int n = job.n;
        if (nj > 0 && !(good = __all_sync(0xffffffffu, wait_apart(&q_empty, (nj - 1) & 1, abort_p)))) break;
        if (n == 0) {
          // q_full's and q_empty's phases go by jobs: an empty one passes its turn on.  `want` comes last: the product
          // warps skip this phase of q_full, so it has to be over before there is a next job to wait for.
          if (lane == 0) {
            mbar_arrive(&q_full);
            mbar_arrive(&q_empty);
            mbar_arrive(&q_empty);
            mbar_arrive(&want);
          }
        } else {
          if (lane == 0) {
            mbar_expect_tx(&q_full, 2 * Smem::kQ);
            for (int t = 0; t < 2; ++t)
              for (int h = 0; h < HD / 64; ++h)
                tma_load_3d(qs + t * Smem::kQ + h * (kTile * 128), &tmQ, h * 64, job.head0, job.q0 + job.tok0 + t * tq, &q_full);
          }
          q_loads = nj + 1;
          // the load of turn w waits for turn w - 4, which waits for its V step, w - 6, to be clean
          dirty_next = job.dirty_from;
          const int first = loads;
          good = load_steps(job, &tmK, ks, 0, [&](int w) {
            if (w == max(0, n - kAhead) && lane == 0) mbar_arrive(&want);
            return clean_steps(jobs[nj & 1], first, w - 5);
          });
          if (good) good = clean_steps(jobs[nj & 1], first, n);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&job_empty[nj & 1]);
      }
      if (good) give_out(Dirty{-1, 0, 0, nullptr});  // no more
    } else if (warp == 10) {
      // ------------------------------------------------------------ loads of V
      bool good = true;
      for (int nj = 0; good; ++nj) {
        if (!(good = __all_sync(0xffffffffu, wait_apart(&job_full[nj & 1], (nj >> 1) & 1, abort_p)))) break;
        const Job job = jobs[nj & 1];
        if (job.lane < 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&job_empty[nj & 1]);
        if (job.n > 0) good = load_steps(job, &tmV, vs, 2, [](int) { return true; });
      }
    } else if (warp == 12) {
      // ------------------------------------------------------------ work
      // the blocks of 2 x tq tokens of 32 lanes at a time; a lane whose rows are out of range has none
      auto blocks_of = [&](int b, bool note) {
        if (b >= p.n_lanes) return 0;
        const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
        if (q0 >= 0 && q1 <= p.n_rows && q1 >= q0) return (q1 - q0 + 2 * tq - 1) / (2 * tq);
        if (note) atomicOr(p.status, kStatusRange);
        return 0;
      };
      int blocks = 0, longest = 0;
      for (int base = 0; base < p.n_lanes; base += 32) {
        blocks += __reduce_add_sync(0xffffffffu, blocks_of(base + lane, blockIdx.x == 0));
        if (base + lane < p.n_lanes) longest = max(longest, p.kv_len[base + lane]);
      }
      longest = __reduce_max_sync(0xffffffffu, longest);
      int scan_base = 0, scan_done = 0;  // items only grow: the scan for a lane goes on where the last one stopped
      // Blocks beyond the last full round over the CTAs are cut into `cut` pieces (a short one into fewer), so that
      // they take less than a round of their own: the least of rounds x (piece + what a piece costs besides).  Not
      // where most blocks are too short for it: every piece that there is not is work taken in vain.
      const int sms = gridDim.x, whole = blocks * subs / sms * sms, rest = blocks * subs - whole;
      int cut = 1;
      float best = 1.0f;
      for (int r = 1; r < 4 && rest > 0; ++r) {
        const int c = min(min(p.pieces, longest / (2 * kPieceSteps * kStep)), min(r * sms, kPromptPieces) / rest);
        const float cost = (float)((rest * c + sms - 1) / sms) * (1.0f / (float)c + 0.05f);
        if (c > 1 && cost < best) {
          cut = c;
          best = cost;
        }
      }
      const int items = whole + rest * cut;
      int item = blockIdx.x;
      bool own = true;  // a CTA's first item is its own
      auto take = [&]() {  // the next job, or one with lane = -1
        Job job = {};
        job.lane = -1;
        for (;;) {
          if (!own) {
            int more = 0;
            if (lane == 0) more = gridDim.x + atomicAdd(p.queue, 1);
            item = __shfl_sync(0xffffffffu, more, 0);
          }
          own = false;
          if (item >= items) break;
          const int over = max(0, item - whole), piece = over % cut, bs = min(item, whole) + over / cut;
          const int most = item < whole ? 1 : cut, sub = bs % subs, blk = bs / subs;
          int b = -1, after = 0;  // the block's lane, the blocks up to its last
          for (; scan_base < p.n_lanes; scan_base += 32) {
            int incl = blocks_of(scan_base + lane, false);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int y = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += y;
            }
            const unsigned has = __ballot_sync(0xffffffffu, blk < scan_done + incl);
            if (has) {
              b = scan_base + __ffs(has) - 1;
              after = scan_done + __shfl_sync(0xffffffffu, incl, __ffs(has) - 1);
              break;
            }
            scan_done += __shfl_sync(0xffffffffu, incl, 31);
          }
          if (b < 0) break;  // only where cu_q decreases and the blocks' count has overflowed
          job.q0 = p.cu_q[b];
          job.n_q = p.cu_q[b + 1] - job.q0;
          job.kv = p.kv_len[b];
          job.seq = p.seqs ? p.seqs[b] : b;
          bool ok = job.seq >= 0 && job.seq < s.max_seqs && job.kv >= 0 && job.kv <= s.max_len();
          if (ok) {
            // every position of the lane has to have a page of the pool
            const int32_t* row = p.table + (size_t)job.seq * s.max_pages;
            const int held = (job.kv + s.page - 1) / s.page;
#pragma unroll 4
            for (int j = lane; j < held; j += 32) {
              const int pg = row[j];
              ok = ok && pg >= 0 && pg < s.n_pages;
            }
          }
          if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) atomicOr(p.status, kStatusRange);
            continue;
          }
          job.tok0 = (after - 1 - blk) * 2 * tq;  // a lane's last block first
          job.head0 = sub * p.pack;
          job.kvh = job.head0 / p.group;
          const int shift = job.kv - job.n_q;
          int n_t[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            // steps a tile needs, by its last token's position
            const int first = job.tok0 + t * tq, last = shift + min(job.n_q, first + tq) - 1;
            n_t[t] = first < job.n_q && last >= 0 ? last / kStep + 1 : 0;
          }
          const int all = max(n_t[0], n_t[1]);
          job.pieces = max(1, min(most, all / kPieceSteps));
          if (piece >= job.pieces) continue;
          const int each = (all + job.pieces - 1) / job.pieces;
          job.piece = piece;
          job.slot = (bs - whole) * cut;
          job.u0 = piece * each;
          job.n = max(0, min(each, all - job.u0));
          for (int t = 0; t < 2; ++t) job.n_t[t] = max(0, min(job.n, n_t[t] - job.u0));
          job.dirty_from = max(0, max(0, shift + job.tok0 + 1) / kStep - job.u0);
          job.lane = b;
          break;
        }
        return job;
      };
      bool good = true;
      for (int nj = 0; good; ++nj) {
        // late, when the job before nears its end: what is taken early is missing where a CTA runs out of work
        if (nj > 0 && !(good = __all_sync(0xffffffffu, wait_apart(&want, (nj - 1) & 1, abort_p)))) break;
        const Job job = take();
        if (nj >= 2 && !(good = __all_sync(0xffffffffu, wait_apart(&job_empty[nj & 1], ((nj >> 1) - 1) & 1, abort_p)))) break;
        if (lane == 0) {
          jobs[nj & 1] = job;
          *(volatile int*)&jobs_taken = nj + 1;
          mbar_arrive(&job_full[nj & 1]);
        }
        __syncwarp();
        if (job.lane < 0) break;
      }
    } else if (warp > 12) {
      // ------------------------------------------------------------ cleaning, with warp 9
      // (a lane's single query behind whole steps leaves nothing to clean, in a call of seconds too)
      for (int g = 0; wait_over_jobs(&go, g & 1, abort_p, &jobs_taken); ++g) {
        const Dirty d = dirt;
        if (d.slot < 0) break;
        clean_step<HD, BF16>(vs + d.slot * Smem::kKv, d, warp - 12);
        mbar_arrive(&clean[d.slot]);
      }
    }
  }

  __syncthreads();
  if (abort_flag) {
    // an abandoned pipeline: neither may products still write TMEM when it is freed, nor loads shared
    // memory when the CTA exits (bounded waits)
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    const long long t0 = clock64();
    if ((warp == 8 || warp == 11) && issued) {
      if (elect_one()) mma_commit(&fin[warp == 11]);
      __syncwarp();
      while (!mbar_try_wait(&fin[warp == 11], 0) && clock64() - t0 < kPWait) {
      }
    }
    if (warp == 9) {
      while (q_loads > 0 && !mbar_try_wait(&q_full, (q_loads - 1) & 1) && clock64() - t0 < kPWait) {
      }
    }
    if (warp == 9 || warp == 10)
      // a slot that only one of the two loaded does not fill: this wait then runs to its limit
      for (int i = max(0, loads - kSlots); i < loads; ++i)
        while (!mbar_try_wait(&full[i % kSlots], (i / kSlots) & 1) && clock64() - t0 < kPWait) {
        }
    __syncthreads();
  }
  if (threadIdx.x == 288 && atomicAdd(p.queue + 1, 1) == (int)gridDim.x - 1) {
    // the last CTA leaves the queue as the next call needs it
    p.queue[0] = 0;
    p.queue[1] = 0;
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

// 16-bit tensor map [z][y][x], row pitches in bytes, box [box_z][box_y][box_x], swizzled by the box's rows (64
// values: 128 bytes, 32: 64).
bool make_tmap3(CUtensorMap* tm, const void* base, bool bf16, uint64_t x, uint64_t y, uint64_t z, uint64_t pitch_y,
                uint64_t pitch_z, uint32_t box_y, uint32_t box_z, uint32_t box_x = 64) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {x, y, z}, strides[2] = {pitch_y, pitch_z};
  const cuuint32_t box[3] = {box_x, box_y, box_z}, estr[3] = {1, 1, 1};
  return enc(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_x == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool BF16>
cudaError_t launch_as(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmO,
                      const PromptParams& p, long long blocks, cudaStream_t st) {
  int limit = 0;
  cudaError_t e = dyn_smem_limit((const void*)paged_prompt_kernel<HD, BF16>, &limit);
  if (e != cudaSuccess) return e;
  if (PromptSmem<HD>::kBytes > limit) return cudaErrorInvalidConfiguration;
  // the kernel's split of registers between its roles needs what it was written for at launch
  static const int regs = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, (const void*)paged_prompt_kernel<HD, BF16>) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs * kPromptThreads < 256 * (kSoftmaxRegs + kOtherRegs)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)min((long long)kSms, blocks * p.pieces));
  cfg.blockDim = dim3(kPromptThreads);
  cfg.dynamicSmemBytes = PromptSmem<HD>::kBytes;
  profile_stream_begin(st);
  e = cudaLaunchKernelEx(&cfg, paged_prompt_kernel<HD, BF16>, tmQ, tmK, tmV, tmO, p);
  profile_stream_end(st);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_prompt(const PagedPromptArgs& a, cudaStream_t st) {
  const PagedShape& s = a.s;
  const size_t off = (size_t)a.layer * s.layer_elems();
  const int group = a.n_heads / s.kv;
  const int pack = prompt_pack(s, a.n_heads);
  const bool bf16 = s.dtype == TL_KV_BF16;
  alignas(64) CUtensorMap tmQ, tmK, tmV, tmO;
  const uint64_t rows = (uint64_t)s.n_pages * s.kv;
  const uint32_t box = s.page < kStep ? s.page : kStep;
  if (!make_tmap3(&tmQ, a.q, bf16, s.hd, a.n_heads, a.n_rows, s.hd * 2, (uint64_t)a.q_stride * 2, pack, kTile / pack) ||
      !make_tmap3(&tmK, a.c.k + off, bf16, s.hd, s.page, rows, s.hd * 2, s.block_elems() * 2, box, 1) ||
      !make_tmap3(&tmV, a.c.v + off, bf16, s.hd, s.page, rows, s.hd * 2, s.block_elems() * 2, box, 1) ||
      !make_tmap3(&tmO, a.out, bf16, s.hd, a.n_heads, a.n_rows, s.hd * 2, (uint64_t)a.n_heads * s.hd * 2,
                  pack < 32 ? pack : 32, pack < 32 ? 32 / pack : 1, 32))
    return cudaErrorInvalidValue;
  const PromptParams p{s,
                       a.c.v + off,
                       a.c.table,
                       a.cu_q,
                       a.kv_len,
                       a.seqs,
                       (uint16_t*)a.out,
                       (uint32_t*)a.ws,
                       (int32_t*)(a.ws + kPagedQueueOff),
                       (int32_t*)(a.ws + 256),
                       (float*)(a.ws + kPagedHead),
                       a.scale * kLog2e,
                       a.n_heads,
                       group,
                       pack,
                       a.n_rows,
                       a.n_lanes,
                       a.plan.pieces};
  if (s.hd == 64)
    return bf16 ? launch_as<64, true>(tmQ, tmK, tmV, tmO, p, a.plan.blocks, st) : launch_as<64, false>(tmQ, tmK, tmV, tmO, p, a.plan.blocks, st);
  return bf16 ? launch_as<128, true>(tmQ, tmK, tmV, tmO, p, a.plan.blocks, st) : launch_as<128, false>(tmQ, tmK, tmV, tmO, p, a.plan.blocks, st);
}

}  // namespace tl
