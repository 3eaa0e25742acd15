// The paged 4-bit KV cache: block tables and slot maps, the writer and the reader (sm_103a).

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.cuh"
#include "kv4.cuh"

namespace cg = cooperative_groups;

namespace lrs {

// ------------------------------------------------------------------------------------------
// Plan: take_i = max(0, need_i - have_i), give_i = max(0, have_i - need_i) and new_i are summed over
// the requests before each one (exclusive prefix sums), which places every page taken, every
// page given back and every token.  One cluster of CTAs does a step in one launch: the lengths
// are read in the first part and written after the cluster's barrier, so in and out may be the
// same arrays; nothing is kept between calls.

constexpr int kPlanThreads = 512;
constexpr int kPlanCluster = 8;

struct PlanReq {
  int have, need, fresh;
  bool bad;
};

__device__ __forceinline__ PlanReq plan_request(const Kv4PlanArgs& a, int i) {
  const int len = a.seq_len[i], keep = a.keep_len ? a.keep_len[i] : len, fresh = a.new_len[i];
  PlanReq r = {0, 0, 0, true};
  if (len < 0 || keep < 0 || keep > len || fresh < 0) return r;
  const long long have = ((long long)len + a.page_len - 1) / a.page_len;
  const long long need = ((long long)keep + fresh + a.page_len - 1) / a.page_len;
  if (have > a.table_stride || (need > a.table_stride && fresh <= a.n_tok)) return r;
  r.bad = false;
  r.have = (int)have;
  r.need = (int)(need > a.table_stride ? have : need);  // more tokens than the slot map holds: refused by the total
  r.fresh = fresh > a.n_tok ? a.n_tok + 1 : fresh;
  return r;
}

__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const Kv4PlanArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), nranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kPlanThreads / 32;
  __shared__ long long wsum[3][NW];
  __shared__ long long total[4];  // this CTA's sums of take, give, new; whether a length is bad

  const int head = a.free_state[0], count = a.free_state[1];
  const int g = rank * kPlanThreads + tid, nthr = nranks * kPlanThreads;
  const int seg = (a.n_seqs + nthr - 1) / nthr;
  const int i0 = min(a.n_seqs, g * seg), i1 = min(a.n_seqs, i0 + seg);
  long long v[3] = {0, 0, 0};
  bool bad = head < 0 || head >= a.ring_len || count < 0 || count > a.ring_len;
  for (int i = i0; i < i1; ++i) {
    const PlanReq r = plan_request(a, i);
    bad |= r.bad;
    v[0] += max(0, r.need - r.have);
    v[1] += max(0, r.have - r.need);
    v[2] += r.fresh;
  }
  long long before[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long s = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    before[k] = s - v[k];
    if (lane == 31) wsum[k][warp] = s;
  }
  const bool any_bad = __syncthreads_or(bad);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long all = 0;
    for (int w = 0; w < NW; ++w) {
      if (w == warp) before[k] += all;
      all += wsum[k][w];
    }
    if (tid == 0) total[k] = all;
  }
  if (tid == 0) total[3] = any_bad;
  cluster.sync();  // every CTA has read the lengths and the ring's state
  long long sum[4] = {0, 0, 0, 0};
  for (int r = 0; r < nranks; ++r) {
    const long long* t = cluster.map_shared_rank(total, r);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long x = t[k];
      if (k < 3 && r < rank) before[k] += x;
      sum[k] += x;
    }
  }
  int status = 0;
  if (sum[3] || count + sum[1] > a.ring_len) status = 2;
  else if (sum[2] > a.n_tok) status = 3;
  else if (sum[0] > count) status = 1;

  if (g == 0) {
    a.status[0] = status;
    a.cu_new[a.n_seqs] = status ? 0 : (int)sum[2];
    a.free_state_out[0] = status ? head : (int)((head + sum[0]) % a.ring_len);
    a.free_state_out[1] = status ? count : (int)(count - sum[0] + sum[1]);
  }
  // pages: few by the lane itself, more by the whole warp
  for (int k = 0; k < seg; ++k) {
    const int i = i0 + k;
    PlanReq r = {0, 0, 0, false};
    if (i < i1) {
      const int len = a.seq_len[i], keep = a.keep_len ? a.keep_len[i] : len;
      if (!status) r = plan_request(a, i);
      a.cu_new[i] = status ? 0 : (int)before[2];
      a.seq_len_out[i] = status ? len : keep + r.fresh;
    }
    const int take = max(0, r.need - r.have), give = max(0, r.have - r.need), n = take + give;
    // taken pages go from the ring's place `at` on to the table from `have`; given ones the other way
    const int at = (int)(take ? (head + before[0]) % a.ring_len : (head + count + before[1]) % a.ring_len);
    const int col = min(r.have, r.need);
    unsigned many = __ballot_sync(0xffffffffu, n > 4);
    if (n <= 4) {
      for (int j = 0; j < n; ++j) {
        int* ring = a.ring + ((long long)at + j) % a.ring_len;
        int* entry = a.table + (long long)i * a.table_stride + col + j;
        if (take) *entry = *ring;
        else *ring = *entry;
      }
    }
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const int wi = __shfl_sync(0xffffffffu, i, src), wn = __shfl_sync(0xffffffffu, n, src);
      const int wat = __shfl_sync(0xffffffffu, at, src), wcol = __shfl_sync(0xffffffffu, col, src);
      const int wtake = __shfl_sync(0xffffffffu, take, src);
      for (int j = lane; j < wn; j += 32) {
        int* ring = a.ring + ((long long)wat + j) % a.ring_len;
        int* entry = a.table + (long long)wi * a.table_stride + wcol + j;
        if (wtake) *entry = *ring;
        else *ring = *entry;
      }
    }
    before[0] += take;
    before[1] += give;
    before[2] += r.fresh;
  }
  cluster.sync();  // table, cu_new and seq_len_out are written
  const int tokens = status ? 0 : (int)sum[2];
  for (int t = g; t < a.n_tok; t += nthr) {
    int slot = -1, pos = -1, lo = -1;
    if (t < tokens) {
      lo = 0;  // the last request that begins at or before t
      for (int hi = a.n_seqs; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_new[mid] <= t) lo = mid;
        else hi = mid;
      }
      pos = a.seq_len_out[lo] - (a.cu_new[lo + 1] - t);
      const int page = a.table[(long long)lo * a.table_stride + pos / a.page_len];
      if (page >= 0 && page < a.n_pages) slot = page * a.page_len + pos % a.page_len;
    }
    a.slot[t] = slot;
    a.pos[t] = pos;
    a.seq[t] = lo;
  }
}

cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const int ncta = a.n_seqs > kPlanThreads || a.n_tok > 4 * kPlanThreads ? kPlanCluster : 1;
  cfg.gridDim = dim3(ncta);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ncta;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_plan_kernel, a);
}

// ------------------------------------------------------------------------------------------
// Append and read.  A lane has four neighbouring dims of a row, so a block of 32 dims is eight
// lanes and its codes are two bytes a lane.

template <typename T>
struct Row4;
template <>
struct Row4<float> {
  static __device__ __forceinline__ float4 load(const float* p) { return *reinterpret_cast<const float4*>(p); }
  static __device__ __forceinline__ void store(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
};
template <>
struct Row4<__half> {
  static __device__ __forceinline__ float4 load(const __half* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  static __device__ __forceinline__ void store(__half* p, float4 v) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t*>(&a);
    u.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = u;
  }
};
template <>
struct Row4<__nv_bfloat16> {
  static __device__ __forceinline__ float4 load(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t*>(&a);
    u.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = u;
  }
};

// Code of x for the scale s (finite, not 0): the nearest integer to x / s, ties to even, plus 8, in
// [0, 15].  n is the rounded product with the reciprocal, at most one off; the remainder x - s n
// is exact wherever it is near s / 2 (s has 11 bits, n four), so comparing it with s / 2 decides.
__device__ __forceinline__ int kv4_code(float x, float s, float inv) {
  float n = rintf(x * inv);
  const float r = fmaf(-n, s, x), h = 0.5f * fabsf(s);
  const bool odd = ((int)n) & 1;
  if (fabsf(r) > h || (fabsf(r) == h && odd)) n += (r > 0.f) == (s > 0.f) ? 1.f : -1.f;
  return (int)fminf(fmaxf(n + 8.f, 0.f), 15.f);
}

// Quantise the four values of this lane with the block's eight lanes: two bytes of codes, the scale's bits.
__device__ __forceinline__ uint32_t kv4_quantise(float4 v, int lane, uint16_t* scale) {
  const float x[4] = {v.x, v.y, v.z, v.w};
  // largest magnitude by the bits of |x|, which order like the values and put NaN above infinity
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  const uint32_t mine = top;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  float m = x[3];
#pragma unroll
  for (int i = 2; i >= 0; --i)
    if ((__float_as_uint(x[i]) & 0x7fffffffu) == mine) m = x[i];  // the lowest index with this lane's largest
  const uint32_t has = __ballot_sync(0xffffffffu, mine == top) & (0xffu << (lane & 24));
  m = __shfl_sync(0xffffffffu, m, __ffs(has) - 1);
  const __half s16 = __float2half_rn(m * -0.125f);
  const float s = __half2float(s16);
  if (!(fabsf(s) <= 65504.f)) {
    *scale = 0x7fffu;  // NaN
    return 0x8888u;
  }
  *scale = __half_as_ushort(s16);
  if (s == 0.f) return 0x8888u;
  const float inv = 1.f / s;
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c |= (uint32_t)kv4_code(x[i], s, inv) << (4 * i);
  return c;
}

constexpr int kRowsThreads = 256;

template <int D, typename T>
__global__ void __launch_bounds__(kRowsThreads) kv4_append_kernel(const Kv4RowsArgs a) {
  constexpr int NB = D / 32, LPR = D / 4;  // lanes per row
  const int lane = threadIdx.x & 31;
  const int heads = a.c.n_kv_heads;
  const long long cap = a.c.n_pages * a.c.page_len;
  const long long rows = (long long)a.n_tok * heads;
  const long long step = (long long)gridDim.x * (kRowsThreads / LPR);
  // whole warps go round together: the quantiser shuffles
  const long long first = ((long long)blockIdx.x * kRowsThreads + (threadIdx.x & ~31)) / LPR;
  for (long long base = first; base < rows; base += step) {
    const long long row = base + lane / LPR;
    const int t = (int)(row / heads), h = (int)(row % heads);
    const int slot = row < rows ? a.slot[t] : -1;
    const bool live = slot >= 0 && slot < cap;
    const int dim = 4 * (lane % LPR), block = dim / 32, l = lane & 7;
    uint8_t* tile = live ? kv4_tile<D>(a.c, slot, h) : nullptr;
    const int p = live ? slot % kKv4Tile : 0;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const T* in = reinterpret_cast<const T*>(side ? a.v_in : a.k_in) + (long long)t * a.row_stride + h * D + dim;
      const float4 x = live ? Row4<T>::load(in) : make_float4(0.f, 0.f, 0.f, 0.f);
      uint16_t scale;
      const uint32_t c = kv4_quantise(x, lane, &scale);
      if (live) {
        uint8_t* part = tile + side * kv4_half(D);
        const int off = side ? kv4_v_off<D>(p, block, l) : kv4_k_off<D>(p, block, l);
        *reinterpret_cast<uint16_t*>(part + off) = (uint16_t)c;
        if (l == 0) *reinterpret_cast<uint16_t*>(part + kv4_codes(D) + (p * NB + block) * 2) = scale;
      }
    }
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kRowsThreads) kv4_read_kernel(const Kv4RowsArgs a) {
  constexpr int NB = D / 32, LPR = D / 4;
  const int heads = a.c.n_kv_heads;
  const long long cap = a.c.n_pages * a.c.page_len;
  const long long n = (long long)a.n_tok * heads * LPR;
  for (long long i = (long long)blockIdx.x * kRowsThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kRowsThreads) {
    const int dim = 4 * (int)(i % LPR), block = dim / 32, l = (dim / 4) & 7;
    const long long row = i / LPR;
    const int t = (int)(row / heads), h = (int)(row % heads);
    const int slot = a.slot[t];
    if (slot < 0 || slot >= cap) continue;
    const uint8_t* tile = kv4_tile<D>(a.c, slot, h);
    const int p = slot % kKv4Tile;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint8_t* part = tile + side * kv4_half(D);
      const int off = side ? kv4_v_off<D>(p, block, l) : kv4_k_off<D>(p, block, l);
      const int c = *reinterpret_cast<const uint16_t*>(part + off);
      const float s = h2f_bits(*reinterpret_cast<const uint16_t*>(part + kv4_codes(D) + (p * NB + block) * 2));
      float4 x;
      x.x = s * (float)((c & 15) - 8);
      x.y = s * (float)((c >> 4 & 15) - 8);
      x.z = s * (float)((c >> 8 & 15) - 8);
      x.w = s * (float)((c >> 12 & 15) - 8);
      Row4<T>::store(reinterpret_cast<T*>(side ? a.v_out : a.k_out) + (long long)t * a.row_stride + h * D + dim, x);
    }
  }
}

static int rows_grid(const Kv4RowsArgs& a, int head_dim) {
  const long long work = (long long)a.n_tok * a.c.n_kv_heads * (head_dim / 4);
  const long long ctas = (work + kRowsThreads - 1) / kRowsThreads;
  return (int)(ctas < (1 << 20) ? ctas : (1 << 20));
}

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, int head_dim, int dtype, cudaStream_t st) {
  const int grid = rows_grid(a, head_dim);
  if (head_dim == 128) {
    if (dtype == KV4_F32) kv4_append_kernel<128, float><<<grid, kRowsThreads, 0, st>>>(a);
    else if (dtype == KV4_F16) kv4_append_kernel<128, __half><<<grid, kRowsThreads, 0, st>>>(a);
    else kv4_append_kernel<128, __nv_bfloat16><<<grid, kRowsThreads, 0, st>>>(a);
  } else {
    if (dtype == KV4_F32) kv4_append_kernel<64, float><<<grid, kRowsThreads, 0, st>>>(a);
    else if (dtype == KV4_F16) kv4_append_kernel<64, __half><<<grid, kRowsThreads, 0, st>>>(a);
    else kv4_append_kernel<64, __nv_bfloat16><<<grid, kRowsThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, int head_dim, int dtype, cudaStream_t st) {
  const int grid = rows_grid(a, head_dim);
  if (head_dim == 128) {
    if (dtype == KV4_F32) kv4_read_kernel<128, float><<<grid, kRowsThreads, 0, st>>>(a);
    else if (dtype == KV4_F16) kv4_read_kernel<128, __half><<<grid, kRowsThreads, 0, st>>>(a);
    else kv4_read_kernel<128, __nv_bfloat16><<<grid, kRowsThreads, 0, st>>>(a);
  } else {
    if (dtype == KV4_F32) kv4_read_kernel<64, float><<<grid, kRowsThreads, 0, st>>>(a);
    else if (dtype == KV4_F16) kv4_read_kernel<64, __half><<<grid, kRowsThreads, 0, st>>>(a);
    else kv4_read_kernel<64, __nv_bfloat16><<<grid, kRowsThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace lrs
