// Rotary positions of query and key heads (include/stage_step.h: stage_op_rope).
//
// Angles.  A position's angle is pos * f radians; only its fraction of a turn matters.  f / 2 pi is taken as a 64-bit
// fraction of a turn (its rounding is f's own, 2^-53 of it), and the product with pos wraps around at whole turns by itself: one
// integer multiplication reduces the angle exactly, at any position.  The top two bits of the fraction (plus an eighth)
// are the quadrant, the rest lies within an eighth of a turn of zero, where float32 holds it to 2^-28 of a turn.
//
// A row is read and written once: the bytes bound it.  A CTA makes its tokens' table of cos and sin in
// shared memory while its first loads are in flight, and every head of the token uses it.
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "step.cuh"

namespace lrs {

namespace {

constexpr int kThreads = 256, kItems = 2;  // items of a thread, all loaded before the table is waited for

// VEC elements as the words that they lie in: taken apart where they are loaded, a thread's loads would wait for one another.
template <typename T, int VEC>
struct Words {
  uint4 q;
};
template <typename T>
struct Words<T, 1> {
  T q;
};
template <typename T, int VEC>
__device__ __forceinline__ void take_apart(const Words<T, VEC>& w, float (&f)[VEC]) {
  T v[VEC];
  memcpy(v, &w, sizeof(v));
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = to_f32(v[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ Words<T, VEC> put_together(const float (&f)[VEC]) {
  T v[VEC];
  Words<T, VEC> w;
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = from_f32<T>(f[i]);
  memcpy(&w, v, sizeof(v));
  return w;
}

// f / 2 pi as a 64-bit fraction of a turn
__device__ __forceinline__ uint64_t turn_of(double f) {
  constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
  double t = f * kTurn;
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}

__device__ __forceinline__ float2 cos_sin_of(int pos, uint64_t turn, float scale) {
  const uint64_t frac = (uint64_t)pos * turn;
  const uint32_t top = (uint32_t)(frac >> 32) + (1u << 29);  // an eighth of a turn up: the quadrant is in the two top bits
  const float x = (float)((int)(top & 0x3FFFFFFFu) - (1 << 29)) * (1.0f / 2147483648.0f);  // in half turns, within +-1/4
  float s, c;
  sincospif(x, &s, &c);
  const uint32_t quad = top >> 30;
  if (quad & 1) {
    const float h = c;
    c = -s;
    s = h;
  }
  if (quad & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c * scale, s * scale);
}

// Division by a number that stays the same: n / d for n < 2^31 (d >= 1), by a multiplication with the rounded-up 2^(32 + s) / d.
struct Div {
  uint32_t d, mul, shift;
};
__host__ Div div_by(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {d, d == 1 ? 0u : (uint32_t)(((1ull << (31 + s)) + d - 1) / d), s == 0 ? 0u : s - 1};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, Div v) { return v.d == 1 ? n : __umulhi(n, v.mul) >> v.shift; }

// An item is two vectors of VEC elements of one head: the halves' parts of VEC pairs, or (interleaved, and dims that are
// only copied) two neighbouring vectors.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const RopeArgs a, int tok_per_cta, int splits, int rot_items,
                                                        Div head_items, Div token_items, Div pairs) {
  extern __shared__ float2 table[];  // [token][rot / 2], and behind it the pairs' turns
  using P = Words<T, VEC>;
  const int t0 = (int)(blockIdx.x / splits) * tok_per_cta, nt = min(tok_per_cta, a.n_tok - t0);
  const int split = (int)(blockIdx.x % splits);
  const int heads = a.hq + a.hk, half = a.rot >> 1;
  const int h0 = (int)((int64_t)heads * split / splits), nh = (int)((int64_t)heads * (split + 1) / splits) - h0;
  const int total = nt * nh * (int)head_items.d;
  uint64_t* turns = reinterpret_cast<uint64_t*>(table + tok_per_cta * half);
  bool have_table = false;

  for (int base = 0; base < total; base += kThreads * kItems) {
    P u[kItems], v[kItems];
    T* out[kItems];
    int d0[kItems], d1[kItems], tok[kItems], pos[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int it = base + i * kThreads + (int)threadIdx.x;
      tok[i] = -1;
      if (it >= total) continue;
      // without splits a token's items are token_items.d
      const int tl = splits == 1 ? (int)quotient(it, token_items) : 0, rest = it - tl * (int)token_items.d;
      const int hl = (int)quotient(rest, head_items), j = rest - hl * (int)head_items.d;
      const int t = t0 + tl, h = h0 + hl;
      const bool is_k = h >= a.hq;
      const int64_t in_off = is_k ? t * a.k_stride + (int64_t)(h - a.hq) * a.head_dim : t * a.q_stride + (int64_t)h * a.head_dim;
      const T* in = static_cast<const T*>(is_k ? a.k : a.q) + in_off;
      const int64_t out_off =
          is_k ? t * a.k_out_stride + (int64_t)(h - a.hq) * a.head_dim : t * a.q_out_stride + (int64_t)h * a.head_dim;
      out[i] = static_cast<T*>(is_k ? a.k_out : a.q_out) + out_off;
      tok[i] = tl;
      pos[i] = a.pos[t];  // looked at below: padding is read like the rest, but not written
      if (INTER) {
        d0[i] = 2 * j * VEC;
        d1[i] = d0[i] + VEC;
      } else if (j < rot_items) {
        d0[i] = j * VEC;
        d1[i] = half + d0[i];
      } else {
        d0[i] = a.rot + 2 * (j - rot_items) * VEC;
        d1[i] = d0[i] + VEC;
      }
      u[i] = *reinterpret_cast<const P*>(in + d0[i]);
      if (d1[i] < a.head_dim) v[i] = *reinterpret_cast<const P*>(in + d1[i]);
    }
    if (!have_table) {
      for (int i = threadIdx.x; i < half; i += kThreads) turns[i] = turn_of(a.freqs[i]);
      __syncthreads();
      for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int tl = (int)quotient(i, pairs);
        table[i] = cos_sin_of(a.pos[t0 + tl], turns[i - tl * half], a.scale);  // of padding: not used
      }
      __syncthreads();
      have_table = true;
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (tok[i] < 0 || pos[i] < 0) continue;
      const float2* cs = table + tok[i] * half;
      float x[VEC], y[VEC];
      if (!INTER || VEC == 1) {  // the pairs are across the two vectors
        if (d0[i] < (INTER ? a.rot : half)) {
          take_apart<T, VEC>(u[i], x);
          take_apart<T, VEC>(v[i], y);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float2 w = cs[INTER ? d0[i] >> 1 : d0[i] + e];
            const float h = x[e];
            x[e] = h * w.x - y[e] * w.y;
            y[e] = y[e] * w.x + h * w.y;
          }
          u[i] = put_together<T, VEC>(x);
          v[i] = put_together<T, VEC>(y);
        }
      } else {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const int d = part ? d1[i] : d0[i];
          if (d >= a.rot) continue;
          take_apart<T, VEC>(part ? v[i] : u[i], x);
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            constexpr int kHi = VEC > 1 ? 1 : 0;
            const float2 w = cs[(d + e) >> 1];
            const float h = x[e];
            x[e] = h * w.x - x[e + kHi] * w.y;
            x[e + kHi] = x[e + kHi] * w.x + h * w.y;
          }
          (part ? v[i] : u[i]) = put_together<T, VEC>(x);
        }
      }
      *reinterpret_cast<P*>(out[i] + d0[i]) = u[i];
      if (d1[i] < a.head_dim) *reinterpret_cast<P*>(out[i] + d1[i]) = v[i];
    }
  }
}

template <typename T, int VEC, bool INTER>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t st) {
  // items of a head: those that turn, and behind them those that are only copied (where something is copied at all)
  const int rot_items = INTER ? (a.rot + 2 * VEC - 1) / (2 * VEC) : a.rot / (2 * VEC);
  const int rest = a.copy ? a.head_dim - a.rot : 0;
  const int head_items = INTER ? ((a.copy ? a.head_dim : a.rot) + 2 * VEC - 1) / (2 * VEC) : rot_items + (rest + 2 * VEC - 1) / (2 * VEC);
  const int heads = a.hq + a.hk, per_tok = heads * head_items;
  // A CTA takes whole tokens, about a round of items, as long as there are some CTAs for each SM; else a token's heads are
  // shared out (each share makes the table for itself).
  const int round = kThreads * kItems;
  int tok_per_cta = std::max(1, std::min(round / std::max(1, per_tok), a.n_tok / 608));
  tok_per_cta = std::min(tok_per_cta, std::max(1, 16384 / (a.rot * 4)));
  int splits = 1;
  if (a.n_tok < 304) splits = std::max(1, std::min({heads, 304 / a.n_tok, (per_tok + kThreads - 1) / kThreads}));
  const size_t smem = (size_t)(tok_per_cta + 1) * (a.rot / 2) * sizeof(float2);
  const int64_t grid = (int64_t)((a.n_tok + tok_per_cta - 1) / tok_per_cta) * splits;
  rope_kernel<T, VEC, INTER><<<(unsigned)grid, kThreads, smem, st>>>(a, tok_per_cta, splits, rot_items, div_by(head_items), div_by(per_tok),
                                                                            div_by(a.rot / 2));
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const RopeArgs& a, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  if (a.interleaved) return a.vec ? launch_t<T, kVec, true>(a, st) : launch_t<T, 1, true>(a, st);
  return a.vec ? launch_t<T, kVec, false>(a, st) : launch_t<T, 1, false>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t st) {
  if (dtype == kTypeF32) return launch_d<float>(a, st);
  if (dtype == kTypeF16) return launch_d<__half>(a, st);
  return launch_d<__nv_bfloat16>(a, st);
}

}  // namespace lrs
