// Product of 8-bit matrices with a float32 scale for each block of 128 (include/stage_step.h: stage_op_f8_gemm).
//
// The scales change along K, so the tensor cores' sums cannot run over all of K: every block of 128 is a product of its own in
// TMEM (four tcgen05.mma of 32), which warps read back, scale by a_scale * w_scale and add to float32 sums in
// registers.  A row of the output lies in one TMEM lane and 128 columns share a weight scale, so a thread's factor is one number
// per block.  Two TMEM buffers: the products of the next block run while this one's are read.
//
// 2048 x 28672 x 4096: 208 us, 2.31 PFLOP/s.  The copies and products alone take 141 us (half the bytes: 121), with the
// buffers handed over 159, read back 174, added up 204: reading and adding is what bounds it, though no unit of it is busy for half
// the time.  Tried on it: columns in two halves with four buffers (292: a product of 128 columns takes as long as one of 256), 16
// warps of sums with 64 columns each (220), 32 TMEM columns at a time (221..231: registers), the factors by asynchronous copies
// (209..216), one commit per block (the same), a lane that waits for its warp (240), waits that ask all the
// time (266); one comparison more in the loop that issues the products takes 237.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>
#include <cuda.h>

#include "common.cuh"
#include "kernels.cuh"
#include "step.cuh"
#include "tc.cuh"

namespace cg = cooperative_groups;

namespace lrs {

namespace {

constexpr uint64_t kWaitNs = 1000000000ull;  // a wait's limit; what misses it is NaN
constexpr uint64_t kDrainNs = 200000000ull;

// A wait with a limit, which also ends as soon as another role of the CTA has given up.  The thread sleeps on the mbarrier (up to the
// hint): one that keeps asking takes shared-memory cycles from the products' operands.
__device__ __forceinline__ bool sleep_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool fwait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  if (sleep_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!sleep_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_ns() - t0 > kWaitNs) {
      *abort_flag = 1;
      if (err) atomicExch(err, 1);
      return false;
    }
  }
  return true;
}

// At a CTA's end: the same with a limit of its own, whoever has given up.
__device__ __forceinline__ bool drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_ns();
  while (!sleep_wait(bar, parity))
    if (global_ns() - t0 > kDrainNs) return false;
  return true;
}

// acc += s * d for two neighbouring columns.  (The same in inline PTX costs a move for each operand: 231 us for 2048 x 28672 x 4096 where
// this takes 202, and single multiply-adds 233.)
__device__ __forceinline__ void fma2(float2& acc, uint32_t d0, uint32_t d1, float2 s) {
  acc = __ffma2_rn(make_float2(__uint_as_float(d0), __uint_as_float(d1)), s, acc);
}

// ---- many rows: tiles of 256 rows x 256 columns, one persistent pair of CTAs per two SMs ----
// A product of a pair reads from each SM's shared memory its 128 rows of a and half of the weights' 256, where two CTAs on their
// own would read all 256 each: with copies coming in at the same time that is more than shared memory gives (and half again
// as much from L2).  Both CTAs: warp 0 copies, warps 4-11 read TMEM and hold the sums (warp w: rows 32 (w % 4) .. + 31 of the CTA's
// 128, columns of half w / 4 - 1).  Warp 1 of the first CTA issues the products.  The first warpgroup gives its registers to the two that
// hold the sums.
constexpr int kBM = 256, kBN = 256, kBK = 128, kThreads = 384;
constexpr int kRegsStart = 168, kRegsRoles = 56, kRegsSums = 224;
static_assert(128 * kRegsRoles + 256 * kRegsSums <= kThreads * kRegsStart, "the warpgroups share out what the block is launched with");

struct Big {
  static constexpr int kStages = 6;
  static constexpr uint32_t kTileA = 128 * kBK, kTileB = 128 * kBK, kStage = kTileA + kTileB;  // of one CTA
  static constexpr uint32_t kOffOut = kStages * kStage;       // 8 warps x 4 KB: rows on their way out
  static constexpr uint32_t kOffBar = kOffOut + 8 * 4096;
  static constexpr uint32_t kSmem = kOffBar + 256 + 1024;
  static constexpr uint32_t kCols = 2 * kBN;
  struct Bars {
    uint64_t full[kStages], empty[kStages], done[2], free_[2];
  };
};

// A warp's 32 rows x COLS columns (row = lane) through 4 KB of shared memory, so that rows leave in whole lines.
template <int COLS, typename T>
__device__ __forceinline__ void store_rows(const float2 (&acc)[COLS / 2], unsigned char* stg, const F8GemmArgs& a, int row0, int col0,
                                           bool ok) {
  constexpr int kPiece = 128 / sizeof(T), kUnit = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  T* y = static_cast<T*>(a.y);
  const float bad = __int_as_float(0x7FC00000);
#pragma unroll
  for (int p = 0; p < COLS / kPiece; ++p) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      union {
        T v[kUnit];
        uint4 q;
      } o;
#pragma unroll
      for (int i = 0; i < kUnit; i += 2) {
        const float2 f = acc[(p * kPiece + u * kUnit + i) / 2];
        o.v[i] = from_f32<T>(ok ? f.x : bad);
        o.v[i + 1] = from_f32<T>(ok ? f.y : bad);
      }
      *reinterpret_cast<uint4*>(stg + lane * 128 + ((u ^ (lane & 7)) << 4)) = o.q;
    }
    __syncwarp();
    const int cp = col0 + p * kPiece;
    if (a.vec) {
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int r = it * 4 + (lane >> 3), u = lane & 7, gm = row0 + r, gn = cp + u * kUnit;
        union {
          T v[kUnit];
          uint4 q;
        } o;
        o.q = *reinterpret_cast<const uint4*>(stg + r * 128 + ((u ^ (r & 7)) << 4));
        if (gm >= a.M) continue;
        T* dst = y + (int64_t)gm * a.y_stride + gn;
        if (gn + kUnit <= a.N) {
          *reinterpret_cast<uint4*>(dst) = o.q;
        } else {
#pragma unroll
          for (int i = 0; i < kUnit; ++i)
            if (gn + i < a.N) dst[i] = o.v[i];
        }
      }
    } else {
      for (int r = 0; r < 32; ++r) {
        const int gm = row0 + r;
#pragma unroll
        for (int c = lane; c < kPiece; c += 32) {
          const T v = *reinterpret_cast<const T*>(stg + r * 128 + (((c / kUnit) ^ (r & 7)) << 4) + (c % kUnit) * sizeof(T));
          if (gm < a.M && cp + c < a.N) y[(int64_t)gm * a.y_stride + cp + c] = v;
        }
      }
    }
    __syncwarp();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    f8_gemm_kernel(const F8GemmArgs a, const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB) {
  using G = Big;
  constexpr int kHalf = kBN / 2;
  extern __shared__ unsigned char raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  G::Bars* B = reinterpret_cast<G::Bars*>(sm + G::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + G::kOffBar + sizeof(G::Bars));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  // S pairs of a cluster share a tile's K blocks; more than one only where a cluster has one tile
  const uint32_t crank = cluster.block_rank(), rank = crank & 1, first = crank & ~1u;
  const int S = (int)cluster.num_blocks() >> 1, share = (int)crank >> 1;
  const int pair = (int)(blockIdx.x >> 1) / S, pairs = (int)(gridDim.x >> 1) / S;
  const int tiles_m = (a.M + kBM - 1) / kBM, tiles = tiles_m * ((a.N + kBN - 1) / kBN);
  const int kb0 = (int)((int64_t)a.nkb * share / S), nkb = (int)((int64_t)a.nkb * (share + 1) / S) - kb0;

  if (tid == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->done[i], 1);
      mbar_init(&B->free_[i], 16);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc_pair(tmem_slot, G::kCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster.sync();  // both CTAs' barriers and TMEM are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    regs_down<kRegsRoles>();
    if (warp == 0 && lane == 0 && a.stall != kStallCopies) {
      int it = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
        const int m0 = tile % tiles_m * kBM + 128 * rank, n0 = tile / tiles_m * kBN + 128 * rank;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % G::kStages;
          if (it >= G::kStages && !(ok = fwait(&B->empty[s], (uint32_t)(it / G::kStages + 1) & 1u, abort_flag, a.error))) break;
          const uint32_t bar = at_rank(&B->full[s], first);  // the first CTA's counts both CTAs' bytes
          if (rank == 0) mbar_arrive_expect_tx(&B->full[s], 2 * G::kStage);
          tma_load_2d_pair(sm + s * G::kStage, &tA, (kb0 + kb) * kBK, m0, bar);
          tma_load_2d_pair(sm + s * G::kStage + G::kTileA, &tB, (kb0 + kb) * kBK, n0, bar);
        }
      }
      // Nothing may still be on its way to shared memory when the CTAs leave, whoever has given up.  The first CTA sees both's copies land;
      // the second one's leaves after it, and where it gave up itself, after a time in which they have.
      if (rank == 0) {
        for (int k = max(0, it - G::kStages); k < it; ++k)
          mbar_wait(&B->full[k % G::kStages], (uint32_t)(k / G::kStages) & 1u, kDrainNs);
      } else if (*abort_flag) {
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
      }
      // The products' last arrivals, which come to both CTAs and which no barrier between these waits for (none comes where somebody gave
      // up; those on `done` are waited for by the warps of the sums).
      for (int k = max(0, it - G::kStages); k < it && !*abort_flag; ++k)
        if (!drain_wait(&B->empty[k % G::kStages], (uint32_t)(k / G::kStages) & 1u)) break;
    } else if (warp == 1 && lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_f8_f32(kBM, kBN);
      int it = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs)
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % G::kStages, d = it & 1;
          if (!(ok = fwait(&B->full[s], (uint32_t)(it / G::kStages) & 1u, abort_flag, a.error))) break;
          if (it >= 2 && !(ok = fwait(&B->free_[d], (uint32_t)(it / 2 + 1) & 1u, abort_flag, a.error))) break;
          tc_fence_after();
          const uint32_t pa = smem_u32(sm + s * G::kStage), pb = pa + G::kTileA;
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk)
            umma_f8_pair(tmem + d * kBN, desc_sw128(pa + kk * 32), desc_sw128(pb + kk * 32), idesc, kk > 0);
          umma_commit_pair(&B->empty[s], first);
          umma_commit_pair(&B->done[d], first);
        }
      // the products finish before TMEM is released, whoever has given up
      if (it > 0) drain_wait(&B->done[(it - 1) & 1], (uint32_t)((it - 1) / 2) & 1u);
    }
  } else {
    regs_up<kRegsSums>();
    const int quarter = warp & 3, half = (warp >> 2) - 1;
    const uint32_t lane_tmem = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(half * kHalf);
    unsigned char* stg = sm + G::kOffOut + (warp - 4) * 4096;
    const uint32_t free0 = at_rank(&B->free_[0], first), free1 = at_rank(&B->free_[1], first);
    int it = 0;
    bool ok = true;
    for (int tile = pair; tile < tiles; tile += pairs) {
      const int m0 = tile % tiles_m * kBM + 128 * rank, n0 = tile / tiles_m * kBN;
      const int row0 = m0 + 32 * quarter, col0 = n0 + half * kHalf;
      const float* sa = a.sa + (int64_t)kb0 * a.sa_stride + min(row0 + lane, a.M - 1);
      const float* sw = a.sw + (int64_t)min(col0 >> 7, (a.N - 1) >> 7) * a.nkb + kb0;
      float2 acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      int blocks = nkb;
      if (a.stall == kStallLate && warp == 4 && tile == pair + pairs) {  // (tests) as if this warp's wait had run out just before its product
        blocks = 0;
        ok = false;
        *abort_flag = 1;
        if (a.error && lane == 0) atomicExch(a.error, 1);
      }
      // the factors of two blocks ahead, multiplied only when they are needed: nothing waits for a load that has just been made
      float fa[2], fw[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = i < blocks ? sa[(int64_t)i * a.sa_stride] : 0.f;
        fw[i] = i < blocks ? sw[i] : 0.f;
      }
#pragma unroll 2
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const int d = it & 1;
        // a warp that has given up once is out of step for good: what is left of its tiles is NaN too
        ok = ok && __all_sync(0xffffffffu, fwait(&B->done[d], (uint32_t)(it / 2) & 1u, abort_flag, a.error));
        if (!ok) break;
        tc_fence_after();
        const float f1 = fa[kb & 1] * fw[kb & 1];
        const float2 f = make_float2(f1, f1);
        if (kb + 2 < blocks) {
          fa[kb & 1] = sa[(int64_t)(kb + 2) * a.sa_stride];
          fw[kb & 1] = sw[kb + 2];
        }
        // 16 columns on their way while the 16 before them are added
        uint32_t r[2][16];
        tmem_ld16(lane_tmem + d * kBN, r[0]);
#pragma unroll
        for (int c = 0; c < kHalf / 16; ++c) {
          tmem_wait_ld16(r[c & 1]);
          if (c + 1 < kHalf / 16) {
            tmem_ld16(lane_tmem + d * kBN + (c + 1) * 16, r[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(d ? free1 : free0);
          }
#pragma unroll
          for (int i = 0; i < 16 / 2; ++i) fma2(acc[c * (16 / 2) + i], r[c & 1][2 * i], r[c & 1][2 * i + 1], f);
        }
      }
      if (S == 1) {
        store_rows<kHalf, T>(acc, stg, a, row0, col0, ok);
      } else {  // the stages' place is free: every copy and product of the tile is done
        float4* row = reinterpret_cast<float4*>(sm) + (32 * quarter + lane) * (kBN / 4);
#pragma unroll
        for (int i = 0; i < kHalf / 4; ++i) {
          const float2 p = acc[2 * i], q = acc[2 * i + 1];
          row[(half * (kHalf / 4) + i) ^ lane] = make_float4(p.x, p.y, q.x, q.y);
        }
      }
    }
  }
  if (S > 1) {  // each CTA adds up its share of its half's rows, the pairs' sums in their order
    __syncthreads();
    cluster.sync();
    bool whole = true;
    for (int j = 0; j < 2 * S; ++j) whole = whole && !*cluster.map_shared_rank(const_cast<int*>(abort_flag), j);
    const int m0 = pair % tiles_m * kBM + 128 * rank, n0 = pair / tiles_m * kBN;
    T* y = static_cast<T*>(a.y);
#pragma unroll 2
    for (int e = tid; e < 128 / S * (kBN / 4); e += kThreads) {
      const int r = 128 / S * share + e / (kBN / 4), u = e % (kBN / 4), gm = m0 + r, gn = n0 + 4 * u;
      if (gm >= a.M || gn >= a.N) continue;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < S; ++j) {
        const float4 p = cluster.map_shared_rank(reinterpret_cast<float4*>(sm), 2 * j + rank)[r * (kBN / 4) + (u ^ (r & 31))];
        v[0] += p.x;
        v[1] += p.y;
        v[2] += p.z;
        v[3] += p.w;
      }
      union {
        T t[4];
        uint2 h;
        uint4 q;
      } o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o.t[i] = from_f32<T>(whole ? v[i] : __int_as_float(0x7FC00000));
      T* dst = y + (int64_t)gm * a.y_stride + gn;
      if (a.vec && gn + 4 <= a.N) {
        if (sizeof(T) == 4)
          *reinterpret_cast<uint4*>(dst) = o.q;
        else
          *reinterpret_cast<uint2*>(dst) = o.h;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (gn + i < a.N) dst[i] = o.t[i];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster.sync();  // the other CTA's products, copies and arrivals are done with this one's memory
  if (warp == 0) tmem_dealloc_pair(tmem, G::kCols);
}

// ---- few rows: 128 weight rows x NT rows of a, the K blocks shared out over a cluster ----
// The weights are what is read, so they are the 128 lanes of the products, once, and the rows of a their columns.  A CTA takes
// a tile of 128 weight rows and its rank's K blocks; the ranks' sums meet in shared memory, added in the order of the ranks.
// Warps 0-3 hold the sums (a weight row per thread), warp 4 copies, warp 5 issues the products.
constexpr int kSmallThreads = 192;

template <int NT, int PER>
struct Small {
  static constexpr int kStages = PER == 3 || NT >= 128 ? 3 : NT == 64 ? 4 : NT == 32 ? 5 : 6;  // PER CTAs per SM
  static constexpr uint32_t kTileW = 128 * kBK, kTileA = NT * kBK, kStage = kTileW + kTileA;
  static constexpr uint32_t kOffScale = kStages * kStage;             // 4 warps x 2 blocks x NT products of scales
  static constexpr uint32_t kOffBar = kOffScale + 4 * 2 * NT * 4;
  static constexpr uint32_t kSmem = kOffBar + 256;
  static constexpr uint32_t kCols = 2 * NT < 32 ? 32 : 2 * NT;
  static_assert(kStages * kStage >= 128 * NT * 4, "the sums take the stages' place");
  struct Bars {
    uint64_t full[kStages], empty[kStages], done[2], free_[2], drain;
  };
};

template <int NT, int PER, typename T>
__global__ void __launch_bounds__(kSmallThreads, PER)
    f8_gemm_small_kernel(const F8GemmArgs a, const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tW) {
  using G = Small<NT, PER>;
  extern __shared__ __align__(1024) unsigned char aligned_raw[];  // (a swizzled tile begins at a multiple of 1024)
  unsigned char* sm = aligned_raw;
  typename G::Bars* B = reinterpret_cast<typename G::Bars*>(sm + G::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + G::kOffBar + sizeof(typename G::Bars));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tile = blockIdx.x / C, n0 = tile * 128;
  const int k0 = (int)((int64_t)a.nkb * rank / C), nk = (int)((int64_t)a.nkb * (rank + 1) / C) - k0;

  if (tid == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->done[i], 1);
      mbar_init(&B->free_[i], 4);
    }
    mbar_init(&B->drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, G::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  float2 acc[NT / 2];
#pragma unroll
  for (int i = 0; i < NT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
  bool ok = true;
  if (warp == 4) {
    if (lane == 0 && a.stall != kStallCopies) {
      int it = 0;
      for (; it < nk; ++it) {
        const int s = it % G::kStages;
        if (it >= G::kStages && !fwait(&B->empty[s], (uint32_t)(it / G::kStages + 1) & 1u, abort_flag, a.error)) break;
        mbar_arrive_expect_tx(&B->full[s], G::kStage);
        tma_load_2d(sm + s * G::kStage, &tW, (k0 + it) * kBK, n0, &B->full[s]);
        tma_load_2d(sm + s * G::kStage + G::kTileW, &tA, (k0 + it) * kBK, 0, &B->full[s]);
      }
      // nothing may still be on its way to shared memory when the CTA leaves, whoever has given up: neither copies nor the products' arrivals
      for (int k = max(0, it - G::kStages); k < it; ++k)
        mbar_wait(&B->full[k % G::kStages], (uint32_t)(k / G::kStages) & 1u, kDrainNs);
      for (int k = max(0, it - G::kStages); k < it && !*abort_flag; ++k)
        if (!drain_wait(&B->empty[k % G::kStages], (uint32_t)(k / G::kStages) & 1u)) break;
    }
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f8_f32(128, NT);
      int it = 0;
      for (; it < nk; ++it) {
        const int s = it % G::kStages, d = it & 1;
        if (!fwait(&B->full[s], (uint32_t)(it / G::kStages) & 1u, abort_flag, a.error)) break;
        if (it >= 2 && !fwait(&B->free_[d], (uint32_t)(it / 2 + 1) & 1u, abort_flag, a.error)) break;
        tc_fence_after();
        const uint32_t pw = smem_u32(sm + s * G::kStage), pa = pw + G::kTileW;
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk)
          umma_f8(tmem + d * NT, desc_sw128(pw + kk * 32), desc_sw128(pa + kk * 32), idesc, kk > 0);
        umma_commit(&B->empty[s]);
        umma_commit(&B->done[d]);
      }
      if (it > 0) {  // the products finish before TMEM is released, whoever has given up
        umma_commit(&B->drain);
        mbar_wait(&B->drain, 0u, kDrainNs);
      }
    }
  } else {
    const uint32_t lane_tmem = tmem + ((uint32_t)(32 * warp) << 16);
    const float* sw = a.sw + (int64_t)tile * a.nkb + k0;
    const float* sa = a.sa + (int64_t)k0 * a.sa_stride;
    float* scales = reinterpret_cast<float*>(sm + G::kOffScale) + warp * 2 * NT;
    constexpr int kPer = (NT + 31) / 32;
    // the next block's factors of columns lane, lane + 32, ..., multiplied only when they are needed
    float next[kPer], next_w = nk > 0 ? sw[0] : 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) next[j] = nk > 0 ? sa[min(lane + 32 * j, a.M - 1)] : 0.f;
    for (int it = 0; it < nk; ++it) {
      const int d = it & 1;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (lane + 32 * j < NT) scales[d * NT + lane + 32 * j] = next[j] * next_w;
      if (it + 1 < nk) {
        next_w = sw[it + 1];
#pragma unroll
        for (int j = 0; j < kPer; ++j) next[j] = sa[(int64_t)(it + 1) * a.sa_stride + min(lane + 32 * j, a.M - 1)];
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, fwait(&B->done[d], (uint32_t)(it / 2) & 1u, abort_flag, a.error));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < NT / 16; ++c) {
        uint32_t r[16];
        tmem_ld16(lane_tmem + d * NT + c * 16, r);
        tmem_wait_ld16(r);
        const float4* f = reinterpret_cast<const float4*>(scales + d * NT + c * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 g = f[i];
          fma2(acc[c * 8 + 2 * i], r[4 * i], r[4 * i + 1], make_float2(g.x, g.y));
          fma2(acc[c * 8 + 2 * i + 1], r[4 * i + 2], r[4 * i + 3], make_float2(g.z, g.w));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->free_[d]);
    }
  }
  const float bad = __int_as_float(0x7FC00000);
  T* y = static_cast<T*>(a.y);
  const bool whole = !*abort_flag;
  if (C == 1) {
    if (warp < 4 && n0 + tid < a.N) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 p = acc[i / 2];
        if (i < a.M) y[(int64_t)i * a.y_stride + n0 + tid] = from_f32<T>(ok && whole ? (i & 1 ? p.y : p.x) : bad);
      }
    }
  } else {
    __syncthreads();  // a CTA that has given up has waited for its copies
    float* sums = reinterpret_cast<float*>(sm);  // [row of a][weight row]
    if (warp < 4) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 p = acc[i / 2];
        if (i < a.M) sums[i * 128 + tid] = ok ? (i & 1 ? p.y : p.x) : bad;
      }
    }
    cluster.sync();
    const int total = a.M * 128, e1 = (int)((int64_t)total * (rank + 1) / C);
    constexpr int kAt = 4;  // values of a thread whose reads of the other CTAs are in flight together
    for (int e = (int)((int64_t)total * rank / C) + tid; e < e1; e += kAt * kSmallThreads) {
      float v[kAt] = {};
      for (int r = 0; r < C; ++r) {
        const float* from = cluster.map_shared_rank(sums, r);
#pragma unroll
        for (int i = 0; i < kAt; ++i) v[i] += e + i * kSmallThreads < e1 ? from[e + i * kSmallThreads] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const int at = e + i * kSmallThreads, n = n0 + (at & 127);
        if (at < e1 && n < a.N) y[(int64_t)(at >> 7) * a.y_stride + n] = from_f32<T>(v[i]);
      }
    }
    cluster.sync();  // the others read these sums until here
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, G::kCols);
}

// ---- up to 16 rows: the weights go from memory to registers ----
// A warp takes 16 weight rows and an eighth of the K blocks, eight warps one after another's; a lane's 32 bytes of a row and block are
// its operands of four mma.sync (m16n8k32, rows of a as the columns): which of the block's K a lane holds does not matter to the
// sum, as long as both operands agree.  No shared memory, TMEM or tensor map comes before the first load, and all of a warp's loads of U
// blocks are in flight together: one row is a matter of latency.
constexpr int kFewWarps = 8;

// The 32 bytes from k on of a row, 0 from K on.
template <bool WIDE>
__device__ __forceinline__ void few_load(const uint8_t* row, int k, int K, uint32_t (&r)[8]) {
  if (k + 32 <= K) {
    if (WIDE) {
      ld_stream_32(row + k, r);
    } else {
      const uint4 x = ld_stream_u4(row + k), y = ld_stream_u4(row + k + 16);
      r[0] = x.x, r[1] = x.y, r[2] = x.z, r[3] = x.w, r[4] = y.x, r[5] = y.y, r[6] = y.z, r[7] = y.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[i] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (k + 4 * i + b < K) r[i] |= (uint32_t)row[k + 4 * i + b] << (8 * b);
    }
  }
}

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int TILES, int U, bool WIDE, typename T>
__global__ void __launch_bounds__(32 * kFewWarps, TILES == 1 ? 3 : TILES == 2 ? 2 : 1) f8_gemm_few_kernel(const F8GemmArgs a) {
  __shared__ float sums[kFewWarps][TILES * 8][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int row0 = blockIdx.x * 16;
  const int k0 = (int)((int64_t)a.nkb * warp / kFewWarps), k1 = (int)((int64_t)a.nkb * (warp + 1) / kFewWarps);
  const uint8_t* w0 = a.w + (int64_t)min(row0 + g, a.N - 1) * a.w_stride;
  const uint8_t* w1 = a.w + (int64_t)min(row0 + g + 8, a.N - 1) * a.w_stride;
  const float* sw = a.sw + (int64_t)(row0 >> 7) * a.nkb;
  float acc[TILES][4];
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;

  for (int kb = k0; kb < k1; kb += U) {
    uint32_t x[U][8], y[U][8], v[U][TILES][8];
    float s[U], f[U][TILES][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = min(kb + u, k1 - 1), k = b * kBK + q * 32;
      few_load<WIDE>(w0, k, a.K, x[u]);
      few_load<WIDE>(w1, k, a.K, y[u]);
      s[u] = sw[b];
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        // columns from M on repeat the last row: nobody reads them
        few_load<WIDE>(a.a + (int64_t)min(t * 8 + g, a.M - 1) * a.a_stride, k, a.K, v[u][t]);
#pragma unroll
        for (int i = 0; i < 2; ++i) f[u][t][i] = a.sa[(int64_t)b * a.sa_stride + min(t * 8 + 2 * q + i, a.M - 1)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + u >= k1) break;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; j += 2) mma_e4m3(d, x[u][j], y[u][j], x[u][j + 1], y[u][j + 1], v[u][t][j], v[u][t][j + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(d[i], f[u][t][i & 1] * s[u], acc[t][i]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][t * 8 + 2 * q + (i & 1)][g + (i & 2 ? 8 : 0)] = acc[t][i];
  __syncthreads();
  const int r = threadIdx.x & 15;
  for (int c = threadIdx.x >> 4; c < min(TILES * 8, a.M); c += 2 * kFewWarps) {
    float out = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) out += sums[w][c][r];
    if (row0 + r < a.N) static_cast<T*>(a.y)[(int64_t)c * a.y_stride + row0 + r] = from_f32<T>(out);
  }
}

template <int TILES, int U, typename T>
cudaError_t launch_few(const F8GemmArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((a.N + 15) / 16);
  const bool wide = !(((uintptr_t)a.a | (uintptr_t)a.w | (uintptr_t)a.a_stride | (uintptr_t)a.w_stride) & 31);
  if (wide)
    f8_gemm_few_kernel<TILES, U, true, T><<<grid, 32 * kFewWarps, 0, st>>>(a);
  else
    f8_gemm_few_kernel<TILES, U, false, T><<<grid, 32 * kFewWarps, 0, st>>>(a);
  return cudaGetLastError();
}

// Once per device: the kernel's shared memory, and whether it has the registers that its warpgroups share out (from a kernel
// with fewer, the one that asks for more would wait forever).
template <typename K>
cudaError_t ready_once(K kernel, size_t smem, int regs, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  if (attr.numRegs < regs) return cudaErrorLaunchOutOfResources;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

template <typename T>
cudaError_t launch_big(const F8GemmArgs& a, cudaStream_t st) {
  using G = Big;
  static_assert(sizeof(G::Bars) + 8 <= 256, "barrier block");
  static_assert(G::kSmem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ready_once(f8_gemm_kernel<T>, G::kSmem, kRegsStart, done);
  if (e != cudaSuccess) return e;
  CUtensorMap tA, tB;
  if (!encode_2d(&tA, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.a_stride, kBK, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tB, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.w_stride, kBK, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  static_assert(G::kStages * G::kStage >= 128 * kBN * 4, "the sums take the stages' place");
  const int64_t tiles = (int64_t)((a.M + kBM - 1) / kBM) * ((a.N + kBN - 1) / kBN);
  const BigSplit split = big_split(tiles, a.nkb, sm_count());
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * split.S * split.clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * split.S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f8_gemm_kernel<T>, a, tA, tB);
}

template <int NT, int PER, typename T>
cudaError_t launch_small_per(const F8GemmArgs& a, cudaStream_t st) {
  using G = Small<NT, PER>;
  static_assert(sizeof(typename G::Bars) + 8 <= 256, "barrier block");
  static_assert(PER * (G::kSmem + 1024) <= 228 * 1024, "shared memory of PER CTAs");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ready_once(f8_gemm_small_kernel<NT, PER, T>, G::kSmem, 0, done);
  if (e != cudaSuccess) return e;
  CUtensorMap tA, tW;
  if (!encode_2d(&tA, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.a_stride, kBK, NT,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.w_stride, kBK, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int tiles = (a.N + 127) / 128;
  // K over a cluster until there are about two CTAs per SM; a power of two, as others leave SMs without a cluster (48 tiles of 32 blocks,
  // 17 rows: 10.8 us with four CTAs, 11.3 with three, 16 with six; 32 tiles of 112 blocks: 15.4 with eight, 16.1 with four)
  int C = 1;
  while (C < 8 && 2 * C * tiles <= 2 * sm_count() && 4 * C <= a.nkb) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * C));
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f8_gemm_small_kernel<NT, PER, T>, a, tA, tW);
}

template <int NT, typename T>
cudaError_t launch_small(const F8GemmArgs& a, cudaStream_t st) {
  // two CTAs per SM with more stages each, or three, where there are weight tiles for more than two (64 rows, 448 tiles of 64 blocks: 92 and
  // 81 us; 250 tiles of 32 blocks: 27 and 34)
  if (NT <= 64 && (a.N + 127) / 128 > 2 * sm_count()) return launch_small_per<NT, NT <= 64 ? 3 : 2, T>(a, st);
  return launch_small_per<NT, 2, T>(a, st);
}

template <typename T>
cudaError_t launch_t(const F8GemmArgs& a, cudaStream_t st) {
  if (a.stall != kStallCopies) {  // (the tests' stalled calls go where there is something to wait for)
    // (8 rows, 57344 x 8192: 72 us, as by weight tiles; one row, 6144 x 4096: 6.7 and 13.  16 rows, whose reads from L2 are as many as the
    // weights': 6144 x 4096 9.6 us, 10.9 by weight tiles; 32000 x 4096 30 and 24.  32 rows: 220 and 80 for 57344 x 8192)
    if (a.M <= 8) return launch_few<1, 2, T>(a, st);
    if (a.M <= 16 && (a.N + 127) / 128 <= sm_count() / 2) return launch_few<2, 2, T>(a, st);
  }
  if (a.M <= 16) return launch_small<16, T>(a, st);
  if (a.M <= 32) return launch_small<32, T>(a, st);
  if (a.M <= 64) return launch_small<64, T>(a, st);
  // up to 128 rows by weight tiles only where few of them share K among eight CTAs (128 x 4096 x 14336: 27 us, 38 in pairs; 128 x 10240 x
  // 8192: 54 and 37)
  if (a.M <= 128 && (a.N + 127) / 128 * 8 <= 2 * sm_count()) return launch_small<128, T>(a, st);
  return launch_big<T>(a, st);
}

}  // namespace

cudaError_t launch_f8_gemm(const F8GemmArgs& a, int y_dtype, cudaStream_t st) {
  if (y_dtype == kTypeF32) return launch_t<float>(a, st);
  if (y_dtype == kTypeF16) return launch_t<__half>(a, st);
  return launch_t<__nv_bfloat16>(a, st);
}

}  // namespace lrs
