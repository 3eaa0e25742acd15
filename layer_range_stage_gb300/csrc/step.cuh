// Launch interface of the step's operators (include/stage_step.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace lrs {

// The types of stage_ops.h: STAGE_F32, STAGE_F16, STAGE_BF16 are 0, 1, 2.
constexpr int kTypeF32 = 0, kTypeF16 = 1, kTypeBf16 = 2;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

struct NormF8Args {
  const void* x = nullptr;
  const void* resid = nullptr;
  void* resid_out = nullptr;
  const float* gamma = nullptr;
  uint8_t* q = nullptr;
  float* scale = nullptr;
  void* y = nullptr;
  int64_t x_stride = 0, resid_stride = 0, resid_out_stride = 0, q_stride = 0, scale_stride = 0, y_stride = 0;
  int n_tok = 0, n = 0;
  float eps = 0.f;
  int vec = 0;  // every row and base at a multiple of four elements
};
cudaError_t launch_norm_f8(const NormF8Args& a, int x_dtype, int resid_dtype, cudaStream_t st);

// For tests: nothing is copied, so that the waits run out; a warp of each CTA gives up on its second tile.
constexpr int kStallCopies = 1, kStallLate = 2;
struct F8GemmArgs {
  const uint8_t* a = nullptr;
  const uint8_t* w = nullptr;
  const float* sa = nullptr;  // [nkb] rows at sa_stride
  const float* sw = nullptr;  // [ceil(N / 128)][nkb]
  void* y = nullptr;
  int* error = nullptr;
  int64_t a_stride = 0, w_stride = 0, sa_stride = 0, y_stride = 0;
  int M = 0, N = 0, K = 0, nkb = 0;
  int vec = 0;  // y's base and rows at multiples of 16 bytes
  int stall = 0;  // tests: kStallCopies or kStallLate
};
// How the product of many rows shares `tiles` tiles of nkb blocks of K out on `sms` SMs: clusters of S pairs of CTAs, which share a tile's K.
struct BigSplit {
  int S;
  unsigned clusters;
};
inline BigSplit big_split(int64_t tiles, int nkb, int sms) {
  const int64_t most = std::max(1, sms / 2);
  // Few tiles: two pairs share one's K (256 x 4096 x 14336, 16 tiles: 38 us, 60 with one; with four pairs, whose clusters of eight SMs do
  // not all find a place at once, 48), unless K is short (256 x 4096 x 2048, 16 blocks: 13.9 us, 13.1 with one; 200 x 1001 x 4096, 32: 17 and
  // 22).  Pairs that share a K have one tile each.
  const int S = tiles <= std::min<int64_t>(32, most) && nkb >= 24 ? 2 : 1;
  return {S, (unsigned)std::min(tiles, most)};
}
cudaError_t launch_f8_gemm(const F8GemmArgs& a, int y_dtype, cudaStream_t st);

struct RopeArgs {
  const void* q = nullptr;
  const void* k = nullptr;
  void* q_out = nullptr;
  void* k_out = nullptr;
  const int* pos = nullptr;
  const double* freqs = nullptr;
  int64_t q_stride = 0, k_stride = 0, q_out_stride = 0, k_out_stride = 0;
  int hq = 0, hk = 0, head_dim = 0, rot = 0, n_tok = 0, interleaved = 0;
  float scale = 1.f;
  int vec = 0;   // bases, strides, heads and pairs allow accesses of 16 bytes (2), or of two elements (1)
  int copy = 0;  // dims from rot on are to be copied (some output is not in place)
};
cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t st);

struct LogprobsArgs {
  const void* z = nullptr;
  const int* tokens = nullptr;
  float* logprob = nullptr;
  float* entropy = nullptr;
  int* rank = nullptr;
  int* top_ids = nullptr;
  float* top_lp = nullptr;
  int64_t stride = 0;
  int rows = 0, vocab = 0, top = 0;
};
constexpr int kLogprobsMaxCluster = 8, kLogprobsMaxChunks = 16384;  // chunks of 32 bytes of a CTA
// CTAs of a row's cluster: as many as `sms` SMs hold without a second wave, of 1024 chunks or more each (64 x 128256: 14 us with four, 22 with
// eight), and as many as a long row needs.
inline int logprobs_cluster(int chunks, int rows, int sms) {
  int C = 1;
  while (C < kLogprobsMaxCluster && ((chunks + C - 1) / C > kLogprobsMaxChunks || (rows * (int64_t)C <= sms && chunks / C >= 1024))) C *= 2;
  return C;
}
cudaError_t launch_logprobs(const LogprobsArgs& a, int dtype, cudaStream_t st);

}  // namespace lrs
