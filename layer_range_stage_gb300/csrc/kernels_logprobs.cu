// Log probabilities from logits (include/stage_step.h: stage_op_logprobs).
//
// A row is read once.  Each thread keeps the largest logit so far, M, the sum S of 2^d with d = (z - M) log2 e, and the sum of
// 2^d d: log p and the entropy follow from them, and two threads' sums merge by scaling with the difference of their M.
//
// The likeliest tokens: the row is cut into chunks of 32 bytes, a thread's load, and a chunk's largest logit (which the running
// maximum needs anyway) is kept in shared memory.  The n_top first tokens lie in the n_top chunks that come first in the same order
// by their largest logit, and those in the n_top threads that come first by theirs.  The n_top-th of the largest of groups of eight
// threads is a bound that few other threads reach (where more do, a search over its bits, a barrier that counts per bit, finds
// one); their chunks above it are ranked by counting, and only the n_top first are read again.
//
// Few rows are split over a cluster's CTAs, whose parts meet in the first one's shared memory.
//
// Many rows are bound by instructions (70 % of the issue slots): 4099 x 32000 in bfloat16 70 us, 3.7 TB/s; about 9 per logit in the loop
// (the exponential unit's share alone would be 26 us), the rest per row.  128 threads a row take as long, 512 take 112 us.  64 x
// 128256 in float32: 14 us; one row of 151936 with 20 alternatives 9.4 us, a chain of dependent steps.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.cuh"
#include "step.cuh"

namespace cg = cooperative_groups;

namespace lrs {

namespace {

constexpr int kTop = 32, kMaxCluster = kLogprobsMaxCluster;
constexpr int kMaxChunks = kLogprobsMaxChunks;  // of a CTA: their maxima take 64 KB
constexpr int kSlack = 16;         // threads above the bound beyond the n_top that are needed, at most
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
// The sums of 2 * FROM neighbouring lanes, in all of them: brought to the largest reference first, then added up.
template <int FROM>
__device__ __forceinline__ Sums merge_lanes(Sums m) {
  float ref = m.ref;
#pragma unroll
  for (int o = FROM; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
  if (m.ref == -INFINITY) {
    m.s = m.t = 0.f;  // nothing, or nothing but masked tokens
  } else {
    const float d = fmaxf((m.ref - ref) * kLog2e, -1000.f), f = ex2(d);
    m.t = f * fmaf(d, m.s, m.t);
    m.s *= f;  // a NaN stays in them
  }
  m.ref = ref;
#pragma unroll
  for (int o = FROM; o > 0; o >>= 1) {
    m.s += __shfl_xor_sync(0xffffffffu, m.s, o);
    m.t += __shfl_xor_sync(0xffffffffu, m.t, o);
  }
  return m;
}

template <typename T>
struct alignas(32) Chunk {
  T v[32 / sizeof(T)];
};

template <int NT>
struct Shared {
  Sums sums[NT / 32];
  int above[NT / 32];
  Sums all;
  int above_all;
  int n_chunks, n_cand;
  uint64_t first_bound;    // 0: none
  uint32_t best_chunk[kTop];
  float bound;             // the last of these chunks' largest logit
  uint64_t list[kTop];     // this CTA's first tokens in order: (ordered logit, ~index)
  uint64_t merged[kTop];
  uint64_t cand[kTop * 16];
};

// Elements of chunk c (of the row's grid of 32-byte chunks, whose first element is -off), -inf outside the row.
template <typename T>
__device__ __forceinline__ void load_chunk(const T* z, int off, int vocab, int c, Chunk<T>& p) {
  constexpr int E = 32 / sizeof(T);
  const int e0 = c * E - off;
  if (e0 >= 0 && e0 + E <= vocab) {
    ld_stream_32(z + e0, reinterpret_cast<uint32_t(&)[8]>(p));
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) p.v[i] = e0 + i >= 0 && e0 + i < vocab ? z[e0 + i] : from_f32<T>(-INFINITY);
  }
}

__device__ __forceinline__ float max_of(const Chunk<float>& p) {
  float top = p.v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) top = max_nan(top, p.v[i]);
  return top;
}
__device__ __forceinline__ float max_of(const Chunk<__half>& p) {
  const __half2* h = reinterpret_cast<const __half2*>(p.v);
  __half2 top = h[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) top = __hmax2_nan(top, h[i]);
  return max_nan(__low2float(top), __high2float(top));
}
__device__ __forceinline__ float max_of(const Chunk<__nv_bfloat16>& p) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(p.v);
  __nv_bfloat162 top = h[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) top = __hmax2_nan(top, h[i]);
  return max_nan(__low2float(top), __high2float(top));
}
__device__ __forceinline__ float2 two_of(const Chunk<float>& p, int i) { return make_float2(p.v[2 * i], p.v[2 * i + 1]); }
__device__ __forceinline__ float2 two_of(const Chunk<__half>& p, int i) {
  return __half22float2(reinterpret_cast<const __half2*>(p.v)[i]);
}
__device__ __forceinline__ float2 two_of(const Chunk<__nv_bfloat16>& p, int i) {
  const uint32_t u = reinterpret_cast<const uint32_t*>(p.v)[i];
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

// NT threads, U chunks of each on their way at once.
template <typename T, bool TOP, int NT, int U>
__global__ void __launch_bounds__(NT) logprobs_kernel(const LogprobsArgs a, int chunks_per_cta) {
  constexpr int E = 32 / sizeof(T);
  extern __shared__ float maxima[];  // [chunks_per_cta], then (8-byte aligned) the chunks above the bound
  __shared__ Shared<NT> sh;
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
  // the next float above zt (of -inf: the lowest number; of the two zeros: the smallest one)
  const float above_zt = unordered(ordered(zt) + 1);
  float ref = -INFINITY, best = -INFINITY;  // the largest logit, and the first chunk of the thread that has it
  int best_at = tid, above = 0;
  float2 s = make_float2(0.f, 0.f), td = s;

  for (int base = tid; base < nc; base += NT * U) {
    Chunk<T> p[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (base + u * NT < nc) load_chunk(z, off, a.vocab, c0 + base + u * NT, p[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = base + u * NT;
      if (c >= nc) break;
      const float top = max_of(p[u]);
      if (TOP) {
        maxima[c] = top;
        if (top > best) {
          best = top;
          best_at = c;
        }
      }
      if (top >= zt) {
        const int e0 = (c0 + c) * E - off;
        if (e0 > t || (e0 >= 0 && e0 + E <= t)) {  // all of the chunk lies on one side of the token: >= before it, > behind
          const float least = e0 > t ? above_zt : zt;
#pragma unroll
          for (int i = 0; i < E; ++i) above += to_f32(p[u].v[i]) >= least;
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const float f = to_f32(p[u].v[i]);
            above += f > zt || (f == zt && e0 + i >= 0 && e0 + i < t) ? 1 : 0;
          }
        }
      }
      if (!(top <= ref)) {  // above, or NaN (which then reaches the sums)
        const float to = top == top ? top : 0.f, d = (ref - to) * kLog2e, g = ex2(d);
        const bool any = ref != -INFINITY;
        const float dd = fmaxf(d, -1000.f);
        td.x = any ? g * fmaf(dd, s.x, td.x) : 0.f;
        td.y = any ? g * fmaf(dd, s.y, td.y) : 0.f;
        s.x = any ? g * s.x : 0.f;
        s.y = any ? g * s.y : 0.f;
        ref = to;
      }
      if (ref == -INFINITY) continue;  // nothing but masked tokens so far
      const float2 down = make_float2(-ref, -ref), l2 = make_float2(kLog2e, kLog2e);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        float2 d = __fmul2_rn(__fadd2_rn(two_of(p[u], i), down), l2), e;
        d.x = max_nan(d.x, -1000.f);  // 2^-1000 is 0 here, and 0 * -1000 too
        d.y = max_nan(d.y, -1000.f);
        e.x = ex2(d.x);
        e.y = ex2(d.y);
        s = __fadd2_rn(s, e);
        td = __ffma2_rn(e, d, td);
      }
    }
  }
  const uint64_t mine = tid < nc ? (uint64_t)ordered(best) << 32 | (uint32_t)~best_at : 0;
  Sums m{ref, s.x + s.y, td.x + td.y};
  m = merge_lanes<16>(m);
  above = __reduce_add_sync(0xffffffffu, above);
  if (lane == 0) {
    sh.sums[warp] = m;
    sh.above[warp] = above;
  }
  if (tid == 0) sh.n_chunks = sh.n_cand = 0;
  if (tid < kTop) sh.list[tid] = 0;
  __syncthreads();
  if (warp == 0) {
    Sums s{-INFINITY, 0.f, 0.f};
    int n = 0;
    if (lane < NT / 32) {
      s = sh.sums[lane];
      n = sh.above[lane];
    }
    s = merge_lanes<NT / 64>(s);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
      sh.all = s;
      sh.above_all = n;
    }
  }
  if (TOP && nc > 0) {
    uint64_t* chunk_list = reinterpret_cast<uint64_t*>(maxima + (chunks_per_cta + 1) / 2 * 2);
    // a bound that at least min(n_top, threads with a chunk) threads' best chunks reach, and few more: the n_top-th of the groups'
    // of eight threads first ...
    uint64_t group = mine;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) group = max(group, __shfl_xor_sync(0xffffffffu, group, o));
    if ((tid & 7) == 0) sh.cand[tid >> 3] = group;
    if (tid == 0) sh.first_bound = 0;
    __syncthreads();
    const int want = min(a.top, min(nc, NT));
    if (tid < NT / 8) {
      const uint64_t key = sh.cand[tid];
      int before = 0;
#pragma unroll 8
      for (int j = 0; j < NT / 8; ++j) before += sh.cand[j] > key;
      if (key && before == want - 1) sh.first_bound = key;
    }
    __syncthreads();
    uint64_t bound = sh.first_bound;
    const int reach = __syncthreads_count(mine >= bound);
    if (bound == 0 || reach > a.top + kSlack) {  // ... or bit by bit, where too many reach that, or there are fewer groups
      bound = 0;
      for (int bit = 63; bit >= 0; --bit) {
        const uint64_t b = bound | 1ull << bit;
        const int n = __syncthreads_count(mine >= b);
        if (n >= want) {
          bound = b;
          if (n <= want + kSlack) break;
        }
      }
    }
    if (mine && mine >= bound) {
      for (int c = tid; c < nc; c += NT) {
        const uint64_t k = (uint64_t)ordered(maxima[c]) << 32 | (uint32_t)~c;
        if (k >= bound) chunk_list[atomicAdd(&sh.n_chunks, 1)] = k;
      }
    }
    __syncthreads();
    const int n_chunks = sh.n_chunks, n_best = min(a.top, n_chunks);
    for (int i = tid; i < n_chunks; i += NT) {
      const uint64_t key = chunk_list[i];
      int before = 0;
      for (int j = 0; j < n_chunks; ++j) before += chunk_list[j] > key;
      if (before < n_best) sh.best_chunk[before] = ~(uint32_t)key;
      if (before == n_best - 1) sh.bound = unordered((uint32_t)(key >> 32));
    }
    __syncthreads();
    // the first of their elements are all among those that reach the last chunk's largest (where there are n_top chunks)
    const float least = n_best == a.top ? sh.bound : -INFINITY;
    for (int i = tid; i < n_best * E; i += NT) {
      const int e = (c0 + (int)sh.best_chunk[i / E]) * E - off + i % E;
      const float f = e >= 0 && e < a.vocab ? to_f32(z[e]) : 0.f;
      if (e >= 0 && e < a.vocab && !(f < least)) sh.cand[atomicAdd(&sh.n_cand, 1)] = (uint64_t)ordered(f) << 32 | (uint32_t)~e;
    }
    __syncthreads();
    const int n_cand = sh.n_cand;
    for (int i = tid; i < n_cand; i += NT) {
      const uint64_t key = sh.cand[i];
      int before = 0;
      for (int j = 0; j < n_cand; ++j) before += sh.cand[j] > key;
      if (before < a.top) sh.list[before] = key;
    }
  }
  if (C > 1)
    cluster.sync();
  else
    __syncthreads();
  if (rank == 0) {
    if (TOP && C > 1) {
      const int n = C * a.top;
      for (int i = tid; i < n; i += NT) sh.cand[i] = cluster.map_shared_rank(&sh, i / a.top)->list[i % a.top];
      __syncthreads();
      for (int i = tid; i < n; i += NT) {
        const uint64_t key = sh.cand[i];
        int before = 0;
        for (int j = 0; j < n; ++j) before += sh.cand[j] > key;
        if (key && before < a.top) sh.merged[before] = key;
      }
      __syncthreads();
    }
    if (tid < 32) {
      Sums s = sh.all;
      int n = sh.above_all;
      if (C > 1) {  // a lane for each CTA, merged in one order
        Sums o{-INFINITY, 0.f, 0.f};
        int k = 0;
        if (lane < C) {
          const Shared<NT>* at = cluster.map_shared_rank(&sh, lane);
          o = at->all;
          k = at->above_all;
        }
        s = merge_lanes<kMaxCluster / 2>(o);
        s.ref = __shfl_sync(0xffffffffu, s.ref, 0);
        s.s = __shfl_sync(0xffffffffu, s.s, 0);
        s.t = __shfl_sync(0xffffffffu, s.t, 0);
        n = __reduce_add_sync(0xffffffffu, k);
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
  if (C > 1) cluster.sync();  // the others' shared memory is read until here
}

template <typename T, bool TOP, int NT, int U>
cudaError_t launch_k(const LogprobsArgs& a, int C, int per, cudaStream_t st) {
  // the bound's threads hold (per + NT - 1) / NT chunks each
  const size_t smem = TOP ? ((size_t)per + 1) / 2 * 8 + (size_t)(a.top + kSlack) * ((per + NT - 1) / NT) * 8 : 0;
  static std::atomic<uint64_t> ready{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(logprobs_kernel<T, TOP, NT, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunks * 4 + (kTop + kSlack) * (kMaxChunks / NT) * 8);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.rows * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, TOP, NT, U>, a, per);
}

template <typename T, bool TOP>
cudaError_t launch_t(const LogprobsArgs& a, cudaStream_t st) {
  constexpr int E = 32 / sizeof(T);
  const int chunks = (a.vocab + E - 1) / E + 1;  // a row that begins inside a chunk has one more
  const int C = logprobs_cluster(chunks, a.rows, sm_count());
  const int per = (chunks + C - 1) / C;
  // one row's latency counts where a cluster shares it: more threads, each with fewer loads after one another
  if (C > 1) return launch_k<T, TOP, 512, 4>(a, C, per, st);
  return launch_k<T, TOP, 256, 2>(a, C, per, st);
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
