// Rotary positions of query and key heads (include/stage_step.h: stage_op_rope).
//
// Angles.  A position's angle is pos * f radians; only its fraction of a turn matters.  f / 2 pi is taken as a 64-bit
// fraction of a turn (its rounding is f's own, 2^-53 of it), and the product with pos wraps around at whole turns by itself: one
// integer multiplication reduces the angle exactly, at any position.  The top two bits of the fraction (plus an eighth)
// are the quadrant, the rest lies within an eighth of a turn of zero, where float32 holds it to 2^-28 of a turn.
//
// A row is read and written once: the bytes bound it.  A warp takes a token's heads (or, where tokens are few, a share of them), a
// lane the same dims of every head it comes to, so that its cos and sin stay in registers; the warp makes the token's table while its
// first heads are on their way.  (With CTAs that went by items of three tokens at a time, a third of the instructions found
// the item's place, and a barrier stood between the loads and the table: 16384 tokens of 40 heads of 128: 82 us, now 65.)
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "kernels.cuh"
#include "step.cuh"

namespace lrs {

namespace {

constexpr int kWarps = 8, kItems = 2;  // heads of a lane that are on their way together (four: 97 us below, for want of registers)

// VEC elements as the words that they lie in: taken apart where they are loaded, a thread's loads would wait for one another.
template <int BYTES>
struct Raw;
template <>
struct Raw<2> {
  uint16_t q;
};
template <>
struct Raw<4> {
  uint32_t q;
};
template <>
struct Raw<8> {
  uint2 q;
};
template <>
struct Raw<16> {
  uint4 q;
};
template <typename T, int VEC>
using Words = Raw<(int)sizeof(T) * VEC>;
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

// f / 2 pi as a 64-bit fraction of a turn (a negative one's by its magnitude: a fraction taken up to its turn would lose f's last bits)
__device__ __forceinline__ uint64_t turn_of(double f) {
  constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
  double t = fabs(f) * kTurn;
  t -= floor(t);
  const uint64_t turn = __double2ull_rn(t * 18446744073709551616.0);
  return f < 0.0 ? 0 - turn : turn;
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

// An item is two vectors of VEC elements of one head: the halves' parts of VEC pairs, or (interleaved, and dims that are
// only copied) two neighbouring vectors.  A token's heads are `chunks` shares of `share` heads.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(32 * kWarps, 4) rope_kernel(const RopeArgs a, int chunks, int share, int rot_items, int head_items) {
  extern __shared__ uint64_t turns[];  // [rot / 2], and behind it a table (cos, sin) [rot / 2] of each warp
  using P = Words<T, VEC>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = a.rot >> 1, heads = a.hq + a.hk;
  float2* table = reinterpret_cast<float2*>(turns + half) + warp * half;
  for (int i = threadIdx.x; i < half; i += 32 * kWarps) turns[i] = turn_of(a.freqs[i]);
  __syncthreads();
  // lanes side by side in a head, and heads side by side in a pass
  const bool narrow = head_items <= 32;
  const int per_pass = narrow ? 32 / head_items : 1;
  const int jl = narrow ? lane % head_items : lane, hl = narrow ? lane / head_items : 0;
  const int64_t units = (int64_t)a.n_tok * chunks, stride = (int64_t)gridDim.x * kWarps;

  for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < units; unit += stride) {
    const int t = (int)(unit / chunks), h0 = (int)(unit - (int64_t)t * chunks) * share, h1 = min(heads, h0 + share);
    const int pos = a.pos[t];
    const T* q = static_cast<const T*>(a.q) + t * a.q_stride;
    const T* k = static_cast<const T*>(a.k) + t * a.k_stride;
    T* q_out = static_cast<T*>(a.q_out) + t * a.q_out_stride;
    T* k_out = static_cast<T*>(a.k_out) + t * a.k_out_stride;
    bool have_table = false;
    for (int jb = 0; jb < head_items; jb += 32) {
      const int j = jb + jl;
      const bool mine = hl < per_pass && j < head_items;
      int d0, d1;
      bool turn0, turn1;  // whether the vectors' dims turn (both or none but where pairs are neighbours)
      if (INTER) {
        d0 = 2 * j * VEC;
        d1 = d0 + VEC;
        turn0 = d0 < a.rot;
        turn1 = VEC == 1 ? turn0 : d1 < a.rot;
      } else {
        turn0 = turn1 = j < rot_items;
        d0 = turn0 ? j * VEC : a.rot + 2 * (j - rot_items) * VEC;
        d1 = d0 + (turn0 ? half : VEC);
      }
      const bool second = d1 < a.head_dim;
      float2 cs[VEC];
      bool have_cs = false;
      for (int hb = h0; hb < h1; hb += per_pass * kItems) {
        P u[kItems], v[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int h = hb + i * per_pass + hl;
          if (!mine || h >= h1) continue;
          const T* in = h < a.hq ? q + h * a.head_dim : k + (h - a.hq) * a.head_dim;
          u[i] = *reinterpret_cast<const P*>(in + d0);
          if (second) v[i] = *reinterpret_cast<const P*>(in + d1);
        }
        if (!have_table) {
          __syncwarp();  // the token before this one is done with it
          if (pos >= 0)
            for (int i = lane; i < half; i += 32) table[i] = cos_sin_of(pos, turns[i], a.scale);
          __syncwarp();
          have_table = true;
        }
        if (pos < 0) continue;  // padding was read like the rest, but is not written
        if (!have_cs) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const int at = !INTER ? d0 + e : VEC == 1 ? d0 >> 1 : ((e < VEC / 2 ? d0 : d1) >> 1) + e % ((VEC + 1) / 2);
            cs[e] = mine && (e < (VEC + 1) / 2 || !INTER ? turn0 : turn1) ? table[at] : make_float2(1.f, 0.f);
          }
          have_cs = true;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int h = hb + i * per_pass + hl;
          if (!mine || h >= h1) continue;
          T* out = h < a.hq ? q_out + h * a.head_dim : k_out + (h - a.hq) * a.head_dim;
          float x[VEC], y[VEC];
          if (!INTER || VEC == 1) {  // the pairs are across the two vectors
            if (turn0) {
              take_apart<T, VEC>(u[i], x);
              take_apart<T, VEC>(v[i], y);
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const float w = x[e];
                x[e] = w * cs[e].x - y[e] * cs[e].y;
                y[e] = y[e] * cs[e].x + w * cs[e].y;
              }
              u[i] = put_together<T, VEC>(x);
              v[i] = put_together<T, VEC>(y);
            }
          } else {
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (!(part ? turn1 : turn0)) continue;
              take_apart<T, VEC>(part ? v[i] : u[i], x);
#pragma unroll
              for (int e = 0; e < VEC / 2; ++e) {
                const float2 c = cs[part * (VEC / 2) + e];
                const float w = x[2 * e];
                x[2 * e] = w * c.x - x[2 * e + 1] * c.y;
                x[2 * e + 1] = x[2 * e + 1] * c.x + w * c.y;
              }
              (part ? v[i] : u[i]) = put_together<T, VEC>(x);
            }
          }
          *reinterpret_cast<P*>(out + d0) = u[i];
          if (second) *reinterpret_cast<P*>(out + d1) = v[i];
        }
      }
    }
  }
}

template <typename T, int VEC, bool INTER>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t st) {
  // items of a head: those that turn, and behind them those that are only copied (where something is copied at all)
  const int rot_items = INTER ? (a.rot + 2 * VEC - 1) / (2 * VEC) : a.rot / (2 * VEC);
  const int rest = a.copy ? a.head_dim - a.rot : 0;
  const int head_items = INTER ? ((a.copy ? a.head_dim : a.rot) + 2 * VEC - 1) / (2 * VEC) : rot_items + (rest + 2 * VEC - 1) / (2 * VEC);
  const int heads = a.hq + a.hk, per_pass = head_items <= 32 ? 32 / head_items : 1;
  // shares of whole passes, as many as it takes for every SM to have its warps
  const int sms = sm_count(), passes = (heads + per_pass - 1) / per_pass;
  const int want = (int)std::min<int64_t>(passes, std::max<int64_t>(1, (int64_t)sms * 2 * kWarps / a.n_tok));
  const int share = (passes + want - 1) / want * per_pass, chunks = (heads + share - 1) / share;
  const size_t smem = (size_t)(kWarps + 1) * (a.rot / 2) * sizeof(float2);
  const int64_t ctas = ((int64_t)a.n_tok * chunks + kWarps - 1) / kWarps;
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, (int64_t)sms * 4);
  rope_kernel<T, VEC, INTER><<<grid, 32 * kWarps, smem, st>>>(a, chunks, share, rot_items, head_items);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const RopeArgs& a, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  // (8000 tokens of 36 heads of 80, 20 of them turned, bf16: 64 us by twos, 68 one by one)
  if (a.interleaved)
    return a.vec == 2 ? launch_t<T, kVec, true>(a, st) : a.vec == 1 ? launch_t<T, 2, true>(a, st) : launch_t<T, 1, true>(a, st);
  return a.vec == 2 ? launch_t<T, kVec, false>(a, st) : a.vec == 1 ? launch_t<T, 2, false>(a, st) : launch_t<T, 1, false>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t st) {
  if (dtype == kTypeF32) return launch_d<float>(a, st);
  if (dtype == kTypeF16) return launch_d<__half>(a, st);
  return launch_d<__nv_bfloat16>(a, st);
}

}  // namespace lrs
