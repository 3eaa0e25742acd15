// Product of 8-bit matrices with a float32 scale for each block of 128 (include/stage_step.h: stage_op_f8_gemm).
//
// The scales change along K, so the tensor cores' sums cannot run over all of K: every block of 128 is a product of its own in
// TMEM (four tcgen05.mma of 32), which warps read back, scale by a_scale * w_scale and add to float32 sums in
// registers.  A row of the output lies in one TMEM lane and 128 columns share a weight scale, so a thread's factor is one number
// per block.  Two TMEM buffers: the products of the next block run while this one's are read.
#include <algorithm>
#include <atomic>

#include <cuda.h>

#include "common.cuh"
#include "kernels.cuh"
#include "step.cuh"
#include "tc.cuh"

namespace lrs {

namespace {

constexpr uint64_t kWaitNs = 1000000000ull;  // a wait's limit; what misses it is NaN
constexpr uint64_t kDrainNs = 200000000ull;

__device__ __forceinline__ bool fwait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_ns() - t0 > kWaitNs) {
      *abort_flag = 1;
      if (err) atomicExch(err, 1);
      return false;
    }
  }
  return true;
}

// acc += s * d for two neighbouring columns
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t s) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(s));
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}

// ---- many rows: tiles of 128 rows x BN columns, one persistent CTA per SM ----
// Warps 0-7 read TMEM and hold the sums (warp w: rows 32 (w % 4) .. + 31, columns of half w / 4), warp 8 copies, warp 9 issues
// the products.
constexpr int kBM = 128, kBK = 128, kThreads = 320;

template <int BN>
struct Big {
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr uint32_t kTileA = kBM * kBK, kTileB = BN * kBK, kStage = kTileA + kTileB;
  static constexpr uint32_t kOffOut = kStages * kStage;       // 8 warps x 4 KB: rows on their way out
  static constexpr uint32_t kOffBar = kOffOut + 8 * 4096;
  static constexpr uint32_t kSmem = kOffBar + 256 + 1024;
  static constexpr uint32_t kCols = 2 * BN;
  struct Bars {
    uint64_t full[kStages], empty[kStages], done[2], free_[2], drain;
  };
};

// A warp's 32 rows x COLS columns (row = lane) through 4 KB of shared memory, so that rows leave in whole lines.
template <int COLS, typename T>
__device__ __forceinline__ void store_rows(const uint64_t (&acc)[COLS / 2], unsigned char* stg, const F8GemmArgs& a, int row0, int col0,
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
        const float2 f = unpack2(acc[(p * kPiece + u * kUnit + i) / 2]);
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

template <int BN, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    f8_gemm_kernel(const F8GemmArgs a, const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB) {
  using G = Big<BN>;
  constexpr int kHalf = BN / 2;
  extern __shared__ unsigned char raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  typename G::Bars* B = reinterpret_cast<typename G::Bars*>(sm + G::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + G::kOffBar + sizeof(typename G::Bars));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles_m = (a.M + kBM - 1) / kBM, tiles = tiles_m * ((a.N + BN - 1) / BN), nkb = a.nkb;

  if (tid == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->done[i], 1);
      mbar_init(&B->free_[i], 8);
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

  if (warp == 8) {
    if (lane == 0 && !a.stall) {
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const int m0 = tile % tiles_m * kBM, n0 = tile / tiles_m * BN;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % G::kStages;
          if (it >= G::kStages && !(ok = fwait(&B->empty[s], (uint32_t)(it / G::kStages + 1) & 1u, abort_flag, a.error))) break;
          mbar_arrive_expect_tx(&B->full[s], G::kStage);
          tma_load_2d(sm + s * G::kStage, &tA, kb * kBK, m0, &B->full[s]);
          tma_load_2d(sm + s * G::kStage + G::kTileA, &tB, kb * kBK, n0, &B->full[s]);
        }
      }
      if (*abort_flag)  // nothing may still be landing in shared memory when the CTA leaves
        for (int k = max(0, it - G::kStages); k < it; ++k)
          mbar_wait(&B->full[k % G::kStages], (uint32_t)(k / G::kStages) & 1u, kDrainNs);
    }
  } else if (warp == 9) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f8_f32(kBM, BN);
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x)
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % G::kStages, d = it & 1;
          if (!(ok = fwait(&B->full[s], (uint32_t)(it / G::kStages) & 1u, abort_flag, a.error))) break;
          if (it >= 2 && !(ok = fwait(&B->free_[d], (uint32_t)(it / 2 + 1) & 1u, abort_flag, a.error))) break;
          tc_fence_after();
          const uint32_t pa = smem_u32(sm + s * G::kStage), pb = pa + G::kTileA;
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk)
            umma_f8(tmem + d * BN, desc_sw128(pa + kk * 32), desc_sw128(pb + kk * 32), idesc, kk > 0);
          umma_commit(&B->empty[s]);
          umma_commit(&B->done[d]);
        }
      if (!ok && it > 0) {  // given up: the products already issued finish before TMEM is released
        umma_commit(&B->drain);
        mbar_wait(&B->drain, 0u, kDrainNs);
      }
    }
  } else {
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lane_tmem = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(half * kHalf);
    unsigned char* stg = sm + G::kOffOut + warp * 4096;
    int it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const int m0 = tile % tiles_m * kBM, n0 = tile / tiles_m * BN;
      const int row0 = m0 + 32 * quarter, col0 = n0 + half * kHalf;
      const float* sa = a.sa + min(row0 + lane, a.M - 1);
      const float* sw = a.sw + (int64_t)min(col0 >> 7, (a.N - 1) >> 7) * nkb;
      uint64_t acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = 0;
      float s = sa[0] * sw[0];
      for (int kb = 0; kb < nkb && ok; ++kb, ++it) {
        const float cur = s;
        if (kb + 1 < nkb) s = sa[(int64_t)(kb + 1) * a.sa_stride] * sw[kb + 1];
        const int d = it & 1;
        ok = __all_sync(0xffffffffu, fwait(&B->done[d], (uint32_t)(it / 2) & 1u, abort_flag, a.error));
        if (!ok) break;
        tc_fence_after();
        uint64_t f;
        asm("mov.b64 %0, {%1, %1};" : "=l"(f) : "r"(__float_as_uint(cur)));
#pragma unroll
        for (int c = 0; c < kHalf / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(lane_tmem + d * BN + c * 32, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) fma2(acc[c * 16 + i], r[2 * i], r[2 * i + 1], f);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->free_[d]);
      }
      store_rows<kHalf, T>(acc, stg, a, row0, col0, ok);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, G::kCols);
}

// Once per device: the kernel's shared memory.
template <typename K>
cudaError_t ready_once(K kernel, size_t smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

template <int BN, typename T>
cudaError_t launch_big(const F8GemmArgs& a, cudaStream_t st) {
  using G = Big<BN>;
  static_assert(sizeof(typename G::Bars) + 8 <= 256, "barrier block");
  static_assert(G::kSmem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ready_once(f8_gemm_kernel<BN, T>, G::kSmem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap tA, tB;
  if (!encode_2d(&tA, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.a_stride, kBK, kBM,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tB, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.w_stride, kBK, BN,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)((a.M + kBM - 1) / kBM) * ((a.N + BN - 1) / BN);
  const int grid = (int)std::min<int64_t>(tiles, std::max(1, sm_count()));
  f8_gemm_kernel<BN, T><<<grid, kThreads, G::kSmem, st>>>(a, tA, tB);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const F8GemmArgs& a, cudaStream_t st) {
  return launch_big<256, T>(a, st);
}

}  // namespace

cudaError_t launch_f8_gemm(const F8GemmArgs& a, int y_dtype, cudaStream_t st) {
  if (y_dtype == kTypeF32) return launch_t<float>(a, st);
  if (y_dtype == kTypeF16) return launch_t<__half>(a, st);
  return launch_t<__nv_bfloat16>(a, st);
}

}  // namespace lrs
