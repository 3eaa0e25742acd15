// Attention over the paged 4-bit KV cache (sm_103a).

#include <cfloat>

#include "common.cuh"
#include "kernels.cuh"
#include "kv4.cuh"

namespace lrs {

// A warp has one (token, query head): its lanes hold D / 32 dims each, positions go by one after another
// with a running maximum and sum.
template <typename T>
__device__ __forceinline__ float to_f32(T v) { return (float)v; }

template <int D, typename T>
__global__ void __launch_bounds__(128) kv4_attn_kernel(const Kv4AttnArgs a) {
  constexpr int NB = D / 32, N = D / 32;  // lane l has dims N l .. N l + N - 1
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(w / a.n_q_heads), j = (int)(w % a.n_q_heads);
  if (t >= a.n_tok || t >= a.cu_q[a.n_seqs]) return;
  int lo = 0;  // the last sequence that begins at or before t
  for (int hi = a.n_seqs; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int k_in = t - a.cu_q[lo], c = a.cu_q[lo + 1] - a.cu_q[lo];
  if (k_in < 0 || k_in >= a.max_q) return;
  const long long len = min((long long)min(a.seq_len[lo], a.max_len), (long long)a.table_stride * a.c.page_len);
  const long long last = len - c + k_in;
  const int h = j / (a.n_q_heads / a.c.n_kv_heads);
  float q[N], o[N], m = -INFINITY, sum = 0.f;
  const T* qp = reinterpret_cast<const T*>(a.q) + (long long)t * a.q_stride + j * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = to_f32(qp[i]) * a.scale;
    o[i] = 0.f;
  }
  const int dim = lane * N, block = dim / 32, l = (dim / 4) & 7, sh = 4 * (dim & 3);
  for (long long p = 0; p <= last; ++p) {
    const int page = a.table[(long long)lo * a.table_stride + p / a.c.page_len];
    if (page < 0 || page >= a.c.n_pages) continue;
    const uint8_t* tile = kv4_tile<D>(a.c, page * a.c.page_len + (int)(p % a.c.page_len), h);
    const int in = (int)(p % kKv4Tile);
    const int ck = *reinterpret_cast<const uint16_t*>(tile + kv4_k_off<D>(in, block, l)) >> sh;
    const int cv = *reinterpret_cast<const uint16_t*>(tile + kv4_half(D) + kv4_v_off<D>(in, block, l)) >> sh;
    const float sk = h2f_bits(*reinterpret_cast<const uint16_t*>(tile + kv4_codes(D) + (in * NB + block) * 2));
    const float sv = h2f_bits(*reinterpret_cast<const uint16_t*>(tile + kv4_half(D) + kv4_codes(D) + (in * NB + block) * 2));
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(q[i], sk * (float)((ck >> 4 * i & 15) - 8), s);
    s = warp_sum(s);
    const float top = fmaxf(m, s), keep = expf(m - top), e = expf(s - top);
    sum = sum * keep + e;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(e, sv * (float)((cv >> 4 * i & 15) - 8), o[i] * keep);
    m = top;
  }
  T* out = reinterpret_cast<T*>(a.out) + (long long)t * a.out_stride + j * D + dim;
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = (T)(sum != 0.f ? o[i] / sum : 0.f);
}

size_t kv4_attention_ws_bytes(int, int, int, int, int, int) { return 256; }

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int head_dim, int dtype, cudaStream_t st) {
  const long long warps = (long long)a.n_tok * a.n_q_heads;
  const unsigned grid = (unsigned)((warps + 3) / 4);
  if (head_dim == 128) {
    if (dtype == KV4_F32) kv4_attn_kernel<128, float><<<grid, 128, 0, st>>>(a);
    else if (dtype == KV4_F16) kv4_attn_kernel<128, __half><<<grid, 128, 0, st>>>(a);
    else kv4_attn_kernel<128, __nv_bfloat16><<<grid, 128, 0, st>>>(a);
  } else {
    if (dtype == KV4_F32) kv4_attn_kernel<64, float><<<grid, 128, 0, st>>>(a);
    else if (dtype == KV4_F16) kv4_attn_kernel<64, __half><<<grid, 128, 0, st>>>(a);
    else kv4_attn_kernel<64, __nv_bfloat16><<<grid, 128, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace lrs
