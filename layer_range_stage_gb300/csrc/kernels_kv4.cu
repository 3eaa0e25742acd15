// The paged 4-bit KV cache: block tables and slot maps, the writer and the reader (sm_103a).

#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "kernels.cuh"
#include "kv4.cuh"
#include "kv4_attn.cuh"

namespace cg = cooperative_groups;

namespace lrs {

// ------------------------------------------------------------------------------------------
// Plan: take_i = max(0, need_i - have_i), give_i = max(0, have_i - need_i) and new_i are summed over
// the requests before each one (exclusive prefix sums), which places every page taken, every
// page given back and every token.  A step is bound by the latency of its few dependent reads.  One cluster of CTAs does
// it in one launch: every CTA computes the sums of all requests for itself, in shared memory, and then they share out
// the page moves and the tokens, in warps' shares of neighbours that look their request up once and go on from there -- so
// a request of thousands of pages or tokens is no longer work than as many small ones (1021 requests with 58 thousand
// tokens: 12 us; 16 with a cluster of eight, 20 when every token was searched for by itself and every thread added up all
// warps' sums, 47 when a warp moved a request's pages).  The lengths are read before the cluster's barrier and written after it, so
// in and out may be the same arrays; nothing is kept between calls.

constexpr int kPlanThreads = 1024, kPlanFew = 256;  // threads of a CTA, and of a lone one
constexpr int kPlanCluster = 16, kPlanPortable = 8;  // CTAs; the smaller one where the GPU (or the part of it that is there) has no room
constexpr int kPlanBatch = 4096;  // requests whose sums lie in shared memory at a time

struct PlanReq {
  int have, need, fresh, end;  // pages before and after, new tokens, positions after
  bool bad;
};

__device__ __forceinline__ PlanReq plan_request(const Kv4PlanArgs& a, int i) {
  const int len = a.seq_len[i], keep = a.keep_len ? a.keep_len[i] : len, fresh = a.new_len[i];
  PlanReq r = {0, 0, 0, 0, true};
  if (len < 0 || keep < 0 || keep > len || fresh < 0) return r;
  const int some = min(fresh, a.n_tok + 1);  // more is refused by the total; the sums below fit 32 bits
  const unsigned pl = (unsigned)a.page_len, stride = (unsigned)a.table_stride;
  const unsigned have = ((unsigned)len + pl - 1) / pl, need = ((unsigned)keep + (unsigned)some + pl - 1) / pl;
  if (have > stride || (need > stride && fresh <= a.n_tok) || (unsigned)keep + (unsigned)some > 0x7fffffffu) return r;
  r.bad = false;
  r.have = (int)have;
  r.need = (int)(need > stride ? have : need);
  r.fresh = some;
  r.end = (int)((unsigned)keep + (unsigned)some);
  return r;
}

struct PlanSmem {
  // per request of the batch: the first of its page moves and of its tokens (batch-wide numbers; one more entry), where
  // its pages lie in the ring, the first table column that moves (negative, less one: given back), its positions
  int move[kPlanBatch + 1], token[kPlanBatch + 1], ring[kPlanBatch], col[kPlanBatch], end[kPlanBatch];
  long long part[3][kPlanThreads / 32], all[3];
};

// Sums of v over the block, and over the threads before this one: within warps, then over the warps by each thread, or by
// the first warp where they are many (32 warps' sums, added up by each thread: 8000 cycles; eight: fewer than a barrier).
__device__ __forceinline__ void plan_scan(PlanSmem& sm, const long long (&v)[3], long long (&before)[3], long long (&sum)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  __syncthreads();  // the last scan's parts are read
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long s = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    before[k] = s - v[k];
    if (lane == 31) sm.part[k][warp] = s;
  }
  __syncthreads();
  if (warps <= 8) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      sum[k] = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w == warp) before[k] += sum[k];
        if (w < warps) sum[k] += sm.part[k][w];
      }
    }
    return;
  }
  if (warp == 0) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const long long mine = lane < warps ? sm.part[k][lane] : 0;
      long long s = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      if (lane < warps) sm.part[k][lane] = s - mine;
      if (lane == 31) sm.all[k] = s;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    before[k] += sm.part[k][warp];
    sum[k] = sm.all[k];
  }
}

// The last i in [0, n) with first[i] <= x (first[0] <= x).
__device__ __forceinline__ int plan_find(const int* first, int n, int x) {
  int lo = 0;
  for (int hi = n; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same from an i with first[i] <= x on, where it is near (first[n] > x).
__device__ __forceinline__ int plan_next(const int* first, int n, int i, int x) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (first[i + 1] > x) return i;
    ++i;
  }
  return first[i + 1] > x ? i : i + plan_find(first + i, n - i, x);
}

__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const Kv4PlanArgs a, const Quotient by_page) {
  extern __shared__ __align__(16) unsigned char plan_raw[];
  PlanSmem& sm = *reinterpret_cast<PlanSmem*>(plan_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, nt = blockDim.x, g = (int)cluster.block_rank() * nt + tid;
  const int nthr = (int)cluster.num_blocks() * nt, R = a.ring_len;
  const int head = a.free_state[0], count = a.free_state[1];
  auto wrap = [R](int x) { return x >= R ? x - R : x; };  // a place in the ring, from less than twice its length

  // May the step be done?  Of one batch the sums below say it
  long long total[3] = {0, 0, 0};
  bool bad = head < 0 || head >= R || count < 0 || count > R;
  int status = 0;
  auto decide = [&]() {
    if (__syncthreads_or(bad) || count + total[1] > R) status = 2;
    else if (total[2] > a.n_tok) status = 3;
    else if (total[0] > count) status = 1;
  };
  const bool one = a.n_seqs <= kPlanBatch;
  if (!one) {
    long long v[3] = {0, 0, 0}, before[3];
    for (int i = tid; i < a.n_seqs; i += nt) {
      const PlanReq r = plan_request(a, i);
      bad |= r.bad;
      v[0] += max(0, r.need - r.have);
      v[1] += max(0, r.have - r.need);
      v[2] += r.fresh;
    }
    plan_scan(sm, v, before, total);
    decide();
  }

  int done[3] = {0, 0, 0};  // takes, gives and tokens of the batches before
  for (int b = 0; b < a.n_seqs || b == 0; b += kPlanBatch) {
    const int m = min(kPlanBatch, a.n_seqs - b), seg = (m + nt - 1) / nt;
    const int i0 = min(m, tid * seg), i1 = min(m, i0 + seg);
    long long v[3] = {0, 0, 0}, before[3], sum[3];
    if (!status) {
      for (int i = i0; i < i1; ++i) {
        const PlanReq r = plan_request(a, b + i);
        bad |= r.bad;
        v[0] += max(0, r.need - r.have);
        v[1] += max(0, r.have - r.need);
        v[2] += r.fresh;
      }
    }
    plan_scan(sm, v, before, sum);
    if (one) {
#pragma unroll
      for (int k = 0; k < 3; ++k) total[k] = sum[k];
      decide();
    }
    if (status) {
#pragma unroll
      for (int k = 0; k < 3; ++k) before[k] = sum[k] = 0;
    }
    for (int i = i0; i < i1; ++i) {
      PlanReq r = {0, 0, 0, 0, false};
      if (!status) r = plan_request(a, b + i);
      const int take = max(0, r.need - r.have), give = max(0, r.have - r.need);
      sm.move[i] = (int)(before[0] + before[1]);
      sm.token[i] = (int)before[2];
      if (!status) sm.ring[i] = wrap(head + (take ? done[0] + (int)before[0] : count + done[1] + (int)before[1]));
      sm.col[i] = give ? -1 - r.need : r.have;
      sm.end[i] = status ? a.seq_len[b + i] : r.end;
      before[0] += take;
      before[1] += give;
      before[2] += r.fresh;
    }
    const int moves = (int)(sum[0] + sum[1]), tokens = (int)sum[2];
    if (tid == 0) {
      sm.move[m] = moves;
      sm.token[m] = tokens;
    }
    cluster.sync();  // this batch's lengths (and the ring's state) are read by every CTA

    for (int i = g; i < m; i += nthr) {
      a.seq_len_out[b + i] = sm.end[i];
      a.cu_new[b + i] = done[2] + sm.token[i];
    }
    // Every warp has neighbouring moves, and neighbouring tokens, and goes on from request to request
    const int lane = tid & 31;
    auto share = [&](int n, int* begin, int* end) {
      const int per = (n + nthr - 1) / nthr * 32;
      *begin = (int)min((long long)n, (long long)(g >> 5) * per);
      *end = min(n, *begin + per);
    };
    int x0, x1;
    share(moves, &x0, &x1);
    for (int x = x0 + lane, i = x < x1 ? plan_find(sm.move, m, x) : 0; x < x1; x += 32) {
      i = plan_next(sm.move, m, i, x);
      const int j = x - sm.move[i], col = sm.col[i];
      int* ring = a.ring + wrap(sm.ring[i] + j);
      int* entry = a.table + (long long)(b + i) * a.table_stride + (col < 0 ? -1 - col : col) + j;
      if (col < 0) *ring = *entry;
      else *entry = *ring;
    }
    // a token's page: of the columns that stay, or the ring's (which nobody writes in this step: what is given back goes
    // behind its last page)
    share(tokens, &x0, &x1);
    for (int x = x0 + lane, i = x < x1 ? plan_find(sm.token, m, x) : 0; x < x1; x += 32) {
      i = plan_next(sm.token, m, i, x);
      const int pos = sm.end[i] - (sm.token[i + 1] - x), c = by_page(pos), col = sm.col[i];
      const int page = col < 0 || c < col ? a.table[(long long)(b + i) * a.table_stride + c]
                                          : a.ring[wrap(sm.ring[i] + c - col)];
      const int t = done[2] + x;
      a.slot[t] = page >= 0 && page < a.n_pages ? page * a.page_len + (pos - c * a.page_len) : -1;
      a.pos[t] = pos;
      a.seq[t] = b + i;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) done[k] += (int)sum[k];
    __syncthreads();  // the sums are read
  }
  for (int t = done[2] + g; t < a.n_tok; t += nthr) a.slot[t] = a.pos[t] = a.seq[t] = -1;
  if (g == 0) {
    a.status[0] = status;
    a.cu_new[a.n_seqs] = done[2];
    a.free_state_out[0] = status ? head : wrap(head + (int)total[0]);
    a.free_state_out[1] = status ? count : (int)(count - total[0] + total[1]);
  }
}

cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0}, small{0};  // one bit per device; small: a cluster of kPlanCluster never gets its CTAs
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool first = dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1);
  if (first) {
    e = cudaFuncSetAttribute(kv4_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PlanSmem));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv4_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.dynamicSmemBytes = sizeof(PlanSmem);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  bool fits = !(small.load(std::memory_order_relaxed) >> (dev & 63) & 1);
  if (first) {
    int clusters = 0;
    cfg.gridDim = dim3(kPlanCluster);
    cfg.blockDim = dim3(kPlanThreads);
    attr[0].val.clusterDim.x = kPlanCluster;
    e = cudaOccupancyMaxActiveClusters(&clusters, kv4_plan_kernel, &cfg);
    if (e != cudaSuccess) cudaGetLastError();
    fits = e == cudaSuccess && clusters > 0;
    if (dev < 64) {
      if (!fits) small.fetch_or(1ull << dev, std::memory_order_relaxed);
      ready.fetch_or(1ull << dev, std::memory_order_release);
    }
  }
  // one CTA where it has a few steps at most: a cluster's launch and barrier cost more than they save (64 requests with a token
  // each: 4.1 us, 5.5 in a cluster; 512 tokens: 4.6 and 5.5; 256 with 2048 tokens: 9.3 and 6.0; 1024 with 49 thousand: 58 and 7)
  const int ncta = a.n_seqs > 2 * kPlanFew || a.n_tok > 3 * kPlanFew ? (fits ? kPlanCluster : kPlanPortable) : 1;
  cfg.gridDim = dim3(ncta);
  cfg.blockDim = dim3(ncta > 1 ? kPlanThreads : kPlanFew);
  attr[0].val.clusterDim.x = ncta;
  return cudaLaunchKernelEx(&cfg, kv4_plan_kernel, a, Quotient(a.page_len));
}

// ------------------------------------------------------------------------------------------
// Append and read.  A lane has eight neighbouring dims of a row: 16 bytes of a 16-bit type, one word of K codes, two
// half-words of V codes; a block of 32 dims is four lanes.  A warp has a token (whose slot is taken apart once) and goes
// through its KV heads, 256 / D of them at a time, two such passes in flight; where the tokens alone would leave SMs
// without work, a warp has one pass.

template <typename T>
struct Row8;
template <>
struct Row8<float> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ void values(const uint32_t (&w)[kWords], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
  // Neighbouring lanes swap halves, so that each of the two stores fills whole 32-byte sectors (`live` is the same in both).
  static __device__ __forceinline__ void store(float* p, const float (&v)[8], bool live) {
    const bool odd = threadIdx.x & 1;
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[4 + i], 1);
    if (live) {
      const float4 own = odd ? make_float4(v[4], v[5], v[6], v[7]) : make_float4(v[0], v[1], v[2], v[3]);
      const float4 got = make_float4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<float4*>(odd ? p - 4 : p) = odd ? got : own;      // the even lane's dims
      *reinterpret_cast<float4*>(odd ? p + 4 : p + 8) = odd ? own : got;  // the odd lane's
    }
  }
};
template <>
struct Row8<__half> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void values(const uint32_t (&w)[kWords], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store(__half* p, const float (&v)[8], bool live) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (live) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Row8<__nv_bfloat16> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void values(const uint32_t (&w)[kWords], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8], bool live) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (live) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Of three.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float y;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Quantise the eight values of this lane with the block's four lanes: the codes, eight to a word, and the scale's bits.
// Code of x for the scale s (finite, not 0): the nearest integer to x / s, ties to even, plus 8, in [0, 15].  Adding
// 1.5 * 2^23 to the product with the reciprocal leaves the integer n in the sum's low bits.  The product is off by less
// than 2^-18, so n is the nearest integer unless x / s lies next to a half; there the remainder x - s n, which is exact
// (s has 11 bits, n four), is compared with s / 2.  The sums' bits, shifted four apart and added up, are the eight
// codes and a constant.
__device__ __forceinline__ uint32_t kv4_quantise(const float (&x)[8], int lane, uint16_t* scale) {
  float high = max_nan(x[0], x[1]), low = min_nan(x[0], x[1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    high = max_nan(high, x[i], x[i + 1]);
    low = min_nan(low, x[i], x[i + 1]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    high = max_nan(high, __shfl_xor_sync(0xffffffffu, high, o));
    low = min_nan(low, __shfl_xor_sync(0xffffffffu, low, o));
  }
  float m = high > -low ? high : low;  // NaN stays
  if (__any_sync(0xffffffffu, high == -low && high > 0.f)) {  // both signs of the largest: the lowest index decides
    const float top = fmaxf(high, -low);
    float mine = 0.f;
#pragma unroll
    for (int i = 7; i >= 0; --i)
      if (fabsf(x[i]) == top) mine = x[i];
    const uint32_t has = __ballot_sync(0xffffffffu, mine != 0.f) & (0xfu << (lane & 28));
    const float first = __shfl_sync(0xffffffffu, mine, has ? __ffs(has) - 1 : lane);
    if (high == -low) m = first;
  }
  const __half s16 = __float2half_rn(m * -0.125f);
  float s = __half2float(s16);
  const bool bad = !(fabsf(s) <= 65504.f);
  *scale = bad ? 0x7fffu : __half_as_ushort(s16);
  if (bad) s = 0.f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  if (s == 0.f) inv = 0.f;
  constexpr float kMagic = 12582912.f;
  float t[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    t[i] = fmaf(x[i], inv, kMagic);
    t[i + 1] = fmaf(x[i + 1], inv, kMagic);
    far = max_abs(far, fmaf(kMagic - t[i], s, x[i]), fmaf(kMagic - t[i + 1], s, x[i + 1]));
  }
  const float h = 0.5f * fabsf(s);
  // A normal scale is m / -8 to 2^-11 of itself, so no integer lies below -8; a subnormal one may be further off
  if (!(far <= 0.9998f * h && fabsf(s) >= 6.103515625e-5f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = t[i] - kMagic, r = fmaf(-n, s, x[i]);
      const bool odd = __float_as_uint(t[i]) & 1;
      if (fabsf(r) > h || (fabsf(r) == h && odd)) t[i] += (r > 0.f) == (s > 0.f) ? 1.f : -1.f;
      // all values count as 0 for the scale 0, and for none (NaN and infinities among them)
      t[i] = s == 0.f ? kMagic : fmaxf(t[i], kMagic - 8.f);
    }
  }
  uint32_t c = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    c = c * 16u + __float_as_uint(fminf(t[i], kMagic + 7.f));
  }
  constexpr uint32_t kOnes = 0x11111111u;
  return c - (0x4B400000u - 8u) * kOnes;
}

constexpr int kRowsThreads = 128;

// Where a warp's token lies: its tile of KV head 0 and its position there; the tiles of a page's next KV head are
// `stride` bytes on.  Null for a slot outside the cache.
template <int D>
__device__ __forceinline__ uint8_t* kv4_place(const Kv4Cache& c, int slot, int* p, long long* stride) {
  *p = slot & (kKv4Tile - 1);
  *stride = (long long)(c.page_len / kKv4Tile) * kv4_tile_bytes(D);
  if (slot < 0 || slot >= c.n_pages * c.page_len) return nullptr;
  const int page = slot / c.page_len, in = slot - page * c.page_len;
  return c.data + (long long)page * c.n_kv_heads * *stride + (in / kKv4Tile) * kv4_tile_bytes(D);
}

// A warp per token, eight dims per lane: a row of a KV head is one access, a block's maximum two shuffles.  Bound by the
// quantiser's instructions (20 per value; 70 % of the issue slots): 16411 tokens of 8 heads of 128, bfloat16, 28.6 us for 86 MB,
// 3.0 TB/s.
template <int D, typename T>
__global__ void __launch_bounds__(kRowsThreads) kv4_append_kernel(const Kv4RowsArgs a, int passes) {
  constexpr int NB = D / 32, LPR = D / 8, RPP = 32 / LPR;  // lanes per row, rows per pass
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.n_tok) return;
  int p;
  long long stride;
  uint8_t* tile = kv4_place<D>(a.c, a.slot[t], &p, &stride);
  if (!tile) return;
  const int l8 = lane % LPR, block = l8 >> 2, tig = l8 & 3;
  const int first = blockIdx.y * passes * RPP + lane / LPR;
  const long long at = t * a.row_stride + 8 * l8;
  constexpr int W = Row8<T>::kWords, AHEAD = 16 / W;  // rows of either side that are asked for at once
  for (int i = 0; i < passes; i += AHEAD) {
    uint32_t w[AHEAD][2][W];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int h = first + (i + j) * RPP;
      const bool live = i + j < passes && h < a.c.n_kv_heads;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const uint4* in = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(side ? a.v_in : a.k_in) + at + (long long)h * D);
#pragma unroll
        for (int k = 0; k < W; k += 4) {
          const uint4 u = live ? in[k / 4] : make_uint4(0, 0, 0, 0);
          w[j][side][k] = u.x, w[j][side][k + 1] = u.y, w[j][side][k + 2] = u.z, w[j][side][k + 3] = u.w;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (i + j >= passes) break;  // the same for the whole warp
      const int h = first + (i + j) * RPP;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        float x[8];
        Row8<T>::values(w[j][side], x);
        uint16_t scale;
        const uint32_t c = kv4_quantise(x, lane, &scale);
        if (h < a.c.n_kv_heads) {
          uint8_t* part = tile + h * stride + side * kv4_half(D);
          if (side == 0) {
            *reinterpret_cast<uint32_t*>(part + kv4_k_off<D>(p, block, 2 * tig)) = c;
          } else {
            *reinterpret_cast<uint16_t*>(part + kv4_v_off<D>(p, block, 2 * tig)) = (uint16_t)c;
            *reinterpret_cast<uint16_t*>(part + kv4_v_off<D>(p, block, 2 * tig + 1)) = (uint16_t)(c >> 16);
          }
          if (tig == 0) *reinterpret_cast<uint16_t*>(part + kv4_codes(D) + (p * NB + block) * 2) = scale;
        }
      }
    }
  }
}

// The same split.  Bound by the writes: 16411 tokens of 8 heads of 128 to float32, 27.3 us for 153 MB, 5.6 TB/s.
template <int D, typename T>
__global__ void __launch_bounds__(kRowsThreads) kv4_read_kernel(const Kv4RowsArgs a, int passes) {
  constexpr int NB = D / 32, LPR = D / 8, RPP = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.n_tok) return;
  int p;
  long long stride;
  const uint8_t* tile = kv4_place<D>(a.c, a.slot[t], &p, &stride);
  if (!tile) return;
  const int l8 = lane % LPR, block = l8 >> 2, tig = l8 & 3;
  const int first = blockIdx.y * passes * RPP + lane / LPR;
  const long long at = t * a.row_stride + 8 * l8;
  for (int i = 0; i < passes; i += 4) {
    uint32_t c[4][2] = {};
    uint16_t s[4][2] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int h = first + (i + j) * RPP;
      if (i + j < passes && h < a.c.n_kv_heads) {
        const uint8_t* part = tile + h * stride;
        c[j][0] = *reinterpret_cast<const uint32_t*>(part + kv4_k_off<D>(p, block, 2 * tig));
        s[j][0] = *reinterpret_cast<const uint16_t*>(part + kv4_codes(D) + (p * NB + block) * 2);
        part += kv4_half(D);
        c[j][1] = *reinterpret_cast<const uint16_t*>(part + kv4_v_off<D>(p, block, 2 * tig)) |
                  (uint32_t)*reinterpret_cast<const uint16_t*>(part + kv4_v_off<D>(p, block, 2 * tig + 1)) << 16;
        s[j][1] = *reinterpret_cast<const uint16_t*>(part + kv4_codes(D) + (p * NB + block) * 2);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j >= passes) break;  // the same for the whole warp
      const int h = first + (i + j) * RPP;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const float sc = h2f_bits(s[j][side]);
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = sc * (float)((int)(c[j][side] >> (4 * k) & 15) - 8);
        Row8<T>::store(reinterpret_cast<T*>(side ? a.v_out : a.k_out) + at + (long long)h * D, x, h < a.c.n_kv_heads);
      }
    }
  }
}

// Passes per warp, and the grid: a warp goes through all heads of its token from 4096 tokens on; below, one pass each (8 heads of
// 128, append from bfloat16 and read to float32, us: all heads 3.6 and 2.9 at 64 tokens, 28 and 29 at 16384; one pass each 2.2
// and 1.9, 37 and 31; equal near 4096).
static int rows_passes(const Kv4RowsArgs& a, int head_dim, dim3* grid) {
  const int per = 256 / head_dim, all = (a.c.n_kv_heads + per - 1) / per;
  const int passes = a.n_tok >= 4096 ? all : 1;
  *grid = dim3((unsigned)((a.n_tok + kRowsThreads / 32 - 1) / (kRowsThreads / 32)), (unsigned)((all + passes - 1) / passes));
  return passes;
}

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, int head_dim, int dtype, cudaStream_t st) {
  dim3 grid;
  const int passes = rows_passes(a, head_dim, &grid);
  if (head_dim == 128) {
    if (dtype == KV4_F32) kv4_append_kernel<128, float><<<grid, kRowsThreads, 0, st>>>(a, passes);
    else if (dtype == KV4_F16) kv4_append_kernel<128, __half><<<grid, kRowsThreads, 0, st>>>(a, passes);
    else kv4_append_kernel<128, __nv_bfloat16><<<grid, kRowsThreads, 0, st>>>(a, passes);
  } else {
    if (dtype == KV4_F32) kv4_append_kernel<64, float><<<grid, kRowsThreads, 0, st>>>(a, passes);
    else if (dtype == KV4_F16) kv4_append_kernel<64, __half><<<grid, kRowsThreads, 0, st>>>(a, passes);
    else kv4_append_kernel<64, __nv_bfloat16><<<grid, kRowsThreads, 0, st>>>(a, passes);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, int head_dim, int dtype, cudaStream_t st) {
  dim3 grid;
  const int passes = rows_passes(a, head_dim, &grid);
  if (head_dim == 128) {
    if (dtype == KV4_F32) kv4_read_kernel<128, float><<<grid, kRowsThreads, 0, st>>>(a, passes);
    else if (dtype == KV4_F16) kv4_read_kernel<128, __half><<<grid, kRowsThreads, 0, st>>>(a, passes);
    else kv4_read_kernel<128, __nv_bfloat16><<<grid, kRowsThreads, 0, st>>>(a, passes);
  } else {
    if (dtype == KV4_F32) kv4_read_kernel<64, float><<<grid, kRowsThreads, 0, st>>>(a, passes);
    else if (dtype == KV4_F16) kv4_read_kernel<64, __half><<<grid, kRowsThreads, 0, st>>>(a, passes);
    else kv4_read_kernel<64, __nv_bfloat16><<<grid, kRowsThreads, 0, st>>>(a, passes);
  }
  return cudaGetLastError();
}

}  // namespace lrs
