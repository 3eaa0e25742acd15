// Log probabilities from logits (include/stage_step.h: stage_op_logprobs).
//
// A row is read once.  Each thread keeps the largest logit so far, M, the sum S of 2^d with d = (z - M) log2 e, and the sum of
// 2^d d: log p and the entropy follow from them, and two threads' sums merge by scaling with the difference of their M.
//
// The likeliest tokens: the row is cut into chunks of 32 bytes, a thread's load, and a chunk's largest logit (which the running
// maximum needs anyway) is kept in shared memory.  The n_top first tokens lie in the n_top chunks that come first in the same order
// by their largest logit, so a warp picks those chunks, and only they are read again.
//
// Few rows are split over a cluster's CTAs, whose parts meet in the first one's shared memory.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "common.cuh"
#include "step.cuh"

namespace cg = cooperative_groups;

namespace lrs {

namespace {

constexpr int kThreads = 256, kTop = 32, kMaxCluster = 8;
constexpr int kMaxChunks = 16384;  // of a CTA: their maxima take 64 KB
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN wins
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Floats in their order as unsigned numbers (all above 0 but for NaN of the negative sign).
__device__ __forceinline__ uint32_t ordered(float f) {
  f = f == 0.f ? 0.f : f;  // -0 and 0 are equal
  const uint32_t b = __float_as_uint(f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

struct Sums {
  float ref, s, t;  // with d = (z - ref) log2 e: the sums of 2^d and of 2^d d; ref = -inf: nothing yet
};
__device__ __forceinline__ Sums merge(Sums a, Sums b) {
  if (b.ref > a.ref) {
    const Sums c = a;
    a = b;
    b = c;
  }
  if (b.ref == -INFINITY) return a;
  const float d = (b.ref - a.ref) * kLog2e, f = ex2(d);  // a NaN in either's sums stays in them
  a.s += f * b.s;
  a.t += f > 0.f ? f * (b.t + d * b.s) : 0.f * b.s;
  return a;
}

template <typename T>
struct alignas(32) Chunk {
  T v[32 / sizeof(T)];
};

struct Shared {
  Sums sums[kThreads / 32];
  int above[kThreads / 32];
  Sums all;
  int above_all;
  int n_best;
  uint32_t best_chunk[kTop];
  int n_cand;
  uint64_t cand[kTop * 16];
  uint64_t list[kTop];  // this CTA's first tokens in order: (ordered logit, ~index)
  uint64_t merged[kTop];
};

// Elements of chunk c (of the row's grid of 32-byte chunks, whose first element is -off), -inf outside the row.
template <typename T>
__device__ __forceinline__ void load_chunk(const T* z, int off, int vocab, int c, Chunk<T>& p) {
  constexpr int E = 32 / sizeof(T);
  const int e0 = c * E - off;
  if (e0 >= 0 && e0 + E <= vocab) {
    const uint4* src = reinterpret_cast<const uint4*>(z + e0);
    uint4* dst = reinterpret_cast<uint4*>(&p);
    dst[0] = ld_stream_u4(src);
    dst[1] = ld_stream_u4(src + 1);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) p.v[i] = e0 + i >= 0 && e0 + i < vocab ? z[e0 + i] : from_f32<T>(-INFINITY);
  }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobsArgs a, int chunks_per_cta) {
  constexpr int E = 32 / sizeof(T);
  extern __shared__ uint32_t maxima[];  // [chunks_per_cta], ordered; 0: taken
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* z = static_cast<const T*>(a.z) + (int64_t)row * a.stride;
  const int off = (int)(((uintptr_t)z & 31) / sizeof(T));
  const int chunks = (a.vocab + off + E - 1) / E;
  const int c0 = min(chunks, rank * chunks_per_cta), nc = min(chunks, c0 + chunks_per_cta) - c0;

  const int t = a.tokens ? a.tokens[row] : -1;
  const bool given = t >= 0 && t < a.vocab;
  const float zt = given ? to_f32(z[t]) : INFINITY;
  Sums m{-INFINITY, 0.f, 0.f};
  int above = 0;
  uint64_t mine = 0;  // the thread's best chunk: (ordered maximum, ~chunk)

  for (int c = tid; c < nc; c += kThreads) {
    Chunk<T> p;
    load_chunk(z, off, a.vocab, c0 + c, p);
    float f[E];
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = to_f32(p.v[i]);
    float top = f[0];
#pragma unroll
    for (int i = 1; i < E; ++i) top = max_nan(top, f[i]);
    if (TOP) {
      const uint32_t k = ordered(top);
      maxima[c] = k;
      mine = max(mine, (uint64_t)k << 32 | (uint32_t)~c);
    }
    if (top >= zt) {
      const int e0 = (c0 + c) * E - off;
#pragma unroll
      for (int i = 0; i < E; ++i) above += f[i] > zt || (f[i] == zt && e0 + i >= 0 && e0 + i < t) ? 1 : 0;
    }
    if (top == -INFINITY) continue;
    if (!(top <= m.ref)) {  // above, or NaN (which then reaches the sums)
      const float ref = top == top ? top : 0.f, d = (m.ref - ref) * kLog2e, g = ex2(d);
      m.t = m.ref == -INFINITY ? 0.f : g * (m.t + fmaxf(d, -1000.f) * m.s);
      m.s = m.ref == -INFINITY ? 0.f : g * m.s;
      m.ref = ref;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float d = max_nan((f[i] - m.ref) * kLog2e, -1000.f);  // 2^-1000 is 0 here, and 0 * -1000 too
      const float e = ex2(d);
      m.s += e;
      m.t = fmaf(e, d, m.t);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.ref = __shfl_down_sync(0xffffffffu, m.ref, o);
    b.s = __shfl_down_sync(0xffffffffu, m.s, o);
    b.t = __shfl_down_sync(0xffffffffu, m.t, o);
    m = merge(m, b);
    above += __shfl_down_sync(0xffffffffu, above, o);
  }
  if (lane == 0) {
    sh.sums[warp] = m;
    sh.above[warp] = above;
  }
  uint64_t* entries = reinterpret_cast<uint64_t*>(sh.cand);  // the threads' best chunks, before the candidates take the place
  if (TOP) entries[tid] = mine;
  __syncthreads();
  if (tid == 0) {
    Sums s = sh.sums[0];
    int n = sh.above[0];
    for (int w = 1; w < kThreads / 32; ++w) {
      s = merge(s, sh.sums[w]);
      n += sh.above[w];
    }
    sh.all = s;
    sh.above_all = n;
  }
  if (TOP) {
    if (warp == 0) {  // the first a.top chunks, one after another
      uint64_t e[kThreads / 32];
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) e[i] = entries[i * 32 + lane];
      int n = 0;
      for (; n < min(a.top, nc); ++n) {
        uint64_t best = e[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) best = max(best, e[i]);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
        const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        const int c = (int)~lo, owner = c % kThreads;
        if (lane == 0) {
          sh.best_chunk[n] = (uint32_t)c;
          maxima[c] = 0;
        }
        __syncwarp();
        uint64_t next = 0;  // the owner's best chunk that is left
        for (int j = owner + lane * kThreads; j < nc; j += 32 * kThreads) {
          const uint32_t k = maxima[j];
          if (k) next = max(next, (uint64_t)k << 32 | (uint32_t)~j);
        }
        const uint32_t nhi = __reduce_max_sync(0xffffffffu, (uint32_t)(next >> 32));
        const uint32_t nlo = __reduce_max_sync(0xffffffffu, (uint32_t)(next >> 32) == nhi ? (uint32_t)next : 0u);
        if (lane == (owner & 31)) {
#pragma unroll
          for (int i = 0; i < kThreads / 32; ++i)
            if (i == owner >> 5) e[i] = (uint64_t)nhi << 32 | nlo;
        }
      }
      if (lane == 0) {
        sh.n_best = n;
        sh.n_cand = 0;
      }
    }
    __syncthreads();
    // their elements: all of them are candidates
    const int n_el = sh.n_best * E;
    for (int i = tid; i < n_el; i += kThreads) {
      const int e = (c0 + (int)sh.best_chunk[i / E]) * E - off + i % E;
      if (e >= 0 && e < a.vocab) sh.cand[atomicAdd(&sh.n_cand, 1)] = (uint64_t)ordered(to_f32(z[e])) << 32 | (uint32_t)~e;
    }
    if (tid < kTop) sh.list[tid] = 0;
    __syncthreads();
    const int n_cand = sh.n_cand;
    for (int i = tid; i < n_cand; i += kThreads) {
      const uint64_t key = sh.cand[i];
      int before = 0;
      for (int j = 0; j < n_cand; ++j) before += sh.cand[j] > key;
      if (before < a.top) sh.list[before] = key;
    }
  }
  cluster.sync();
  if (rank == 0) {
    if (TOP && C > 1) {
      for (int i = tid; i < C * kTop; i += kThreads) sh.cand[i] = cluster.map_shared_rank(&sh, i / kTop)->list[i % kTop];
      __syncthreads();
      for (int i = tid; i < C * kTop; i += kThreads) {
        const uint64_t key = sh.cand[i];
        int before = 0;
        for (int j = 0; j < C * kTop; ++j) before += sh.cand[j] > key;
        if (key && before < a.top) sh.merged[before] = key;
      }
      __syncthreads();
    }
    if (tid < 32) {
      Sums s = sh.all;
      int n = sh.above_all;
      for (int r = 1; r < C; ++r) {
        const Shared* o = cluster.map_shared_rank(&sh, r);
        s = merge(s, o->all);
        n += o->above_all;
      }
      const float ls = log2f(s.s);
      const bool bad = !(s.s > 0.f) || !(s.ref < INFINITY);
      if (tid == 0) {
        const float lp = bad || !given ? __int_as_float(0x7FC00000) : (zt - s.ref) - ls * kLn2;
        if (a.logprob) a.logprob[row] = lp;
        if (a.entropy) a.entropy[row] = bad ? __int_as_float(0x7FC00000) : (ls - s.t / s.s) * kLn2;
        if (a.rank) a.rank[row] = bad || !given ? -1 : n;
      }
      if (TOP && tid < a.top) {
        const uint64_t key = C > 1 ? sh.merged[tid] : sh.list[tid];
        if (a.top_ids) a.top_ids[(int64_t)row * a.top + tid] = bad ? -1 : (int)~(uint32_t)key;
        if (a.top_lp)
          a.top_lp[(int64_t)row * a.top + tid] =
              bad ? __int_as_float(0x7FC00000) : (unordered((uint32_t)(key >> 32)) - s.ref) - ls * kLn2;
      }
    }
  }
  cluster.sync();  // the others' shared memory is read until here
}

template <typename T, bool TOP>
cudaError_t launch_t(const LogprobsArgs& a, cudaStream_t st) {
  constexpr int E = 32 / sizeof(T);
  const int chunks = (a.vocab + E - 1) / E + 1;  // a row that begins inside a chunk has one more
  int C = 1;
  while (C < kMaxCluster && ((chunks + C - 1) / C > kMaxChunks || (a.rows * (int64_t)C < 304 && chunks / C >= 1024))) C *= 2;
  const int per = (chunks + C - 1) / C;
  const size_t smem = TOP ? (size_t)per * 4 : 0;
  static std::atomic<uint64_t> ready{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(logprobs_kernel<T, TOP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunks * 4);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, TOP>, a, per);
}

template <typename T>
cudaError_t launch_d(const LogprobsArgs& a, cudaStream_t st) {
  return a.top ? launch_t<T, true>(a, st) : launch_t<T, false>(a, st);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, int dtype, cudaStream_t st) {
  if (dtype == kTypeF32) return launch_d<float>(a, st);
  if (dtype == kTypeF16) return launch_d<__half>(a, st);
  return launch_d<__nv_bfloat16>(a, st);
}

}  // namespace lrs
