// The residual's addition, an RMS norm, and 8-bit rows with scales (include/stage_step.h: stage_op_norm_f8).
//
// One pass: a row's values stay in registers between the sum of squares and the codes.  A warp takes a
// block of 128 columns at a time, four neighbouring columns a lane, so that a block's largest value is one warp
// reduction and its codes are one store of 128 bytes.  The bytes in and out are its floor; what bounds it is the chain from a row's
// loads over its sum to its stores, with 32 warps on an SM: 2048 x 4096 (bfloat16 onto float32) 18 us, 5.1 TB/s; 16411 x 8192 in
// bfloat16 207 us, 4.6 TB/s (its warps' sums and roots are a third of the instructions there; one warp that finishes for the row: 231,
// for its second barrier); float32 255 us, 6.9 TB/s; one row of 4096 2.7 us.  Rows of more than 16384 columns do not fit their registers:
// 4096 x 28672 in bfloat16 99 us without gamma, 3.6 TB/s.
//
// The codes are defined by float32 roundings, so two machines agree if they agree on r = fl(1 / sqrt(mean + eps)).  A float32
// sum would not do: its last bits depend on its order, and where r differs by one unit so does a code now and then.
// The sum is held as an unevaluated pair of float32 (every addition's error is caught exactly and added up: Knuth's
// two-sum), about 2^-45 of it, and r comes from the reciprocal square root by one Newton step whose residual
// 1 - m r^2 is formed in pairs as well, so that its only rounding that counts is the last.  Means beyond 2^+-90, whose squares or root
// leave float32's range on the way, are scaled by a power of two first.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.cuh"
#include "step.cuh"

namespace lrs {

namespace {

struct Pair {  // an unevaluated sum hi + lo
  float hi, lo;
};

__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair r;
  float e;
  two_sum(a.hi, b.hi, r.hi, e);
  r.lo = __fadd_rn(__fadd_rn(a.lo, b.lo), e);
  return r;
}

// sum / n + eps
__device__ __forceinline__ Pair mean_of(Pair sum, float n, float eps) {
  const float q = __fdiv_rn(sum.hi, n);
  const float rem = __fadd_rn(__fmaf_rn(-q, n, sum.hi), sum.lo);
  Pair m;
  float e;
  two_sum(q, eps, m.hi, e);
  m.lo = __fadd_rn(__fdiv_rn(rem, n), e);
  two_sum(m.hi, m.lo, m.hi, m.lo);
  return m;
}
// fl(1 / sqrt(m)) where it lies between these bounds: beyond them m's squares, r^2 or what r^2 leaves out are no float32, and what comes
// out is beyond the bounds too, or NaN
constexpr float kLeastRoot = 0x1p-45f, kMostRoot = 0x1p45f;
__device__ __forceinline__ float recip_root(Pair m) {
  const float r = rsqrtf(m.hi);
  const float p = __fmul_rn(r, r), pe = __fmaf_rn(r, r, -p);
  const float t = __fmul_rn(m.hi, p), te = __fmaf_rn(m.hi, p, -t);
  // 1 - (m.hi + m.lo) (p + pe), t being next to 1
  float d = __fsub_rn(1.f, t);
  d = __fsub_rn(d, te);
  d = __fmaf_rn(-m.hi, pe, d);
  d = __fmaf_rn(-m.lo, p, d);
  return __fmaf_rn(__fmul_rn(0.5f, r), d, r);
}

// The same for two sums side by side; a - b as a multiply-add, which is one packed instruction.
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }
__device__ __forceinline__ void two_sum2(float2 a, float2 b, float2& s, float2& e) {
  s = __fadd2_rn(a, b);
  const float2 t = sub2(s, a);
  e = __fadd2_rn(sub2(a, sub2(s, t)), sub2(b, t));
}

template <typename T>
struct alignas(sizeof(T) * 4) Four {
  T v[4];
};

// Columns of lane's four values in a block: 4 lane + i side by side (VEC: rows at multiples of four elements, and as many), or
// lane + 32 i.

// Four values as the words that they lie in: what is made of them comes later, so that a row's loads do not wait for one another
// (taken apart where they are loaded, they do: 16411 rows of 8192: 390 us).
template <typename T>
struct Words {
  uint32_t w[sizeof(T)];
};
// The four columns from `at` on (VEC), or `at` + 32 i; those from n on are 0.
template <bool VEC, typename T>
__device__ __forceinline__ Words<T> load4(const T* row, int at, int n) {
  Words<T> p;
  if (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) p.w[i] = 0;
    if (at < n) {
      if (sizeof(T) == 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(row + at);
        p.w[0] = q.x;
        p.w[1] = q.y;
        p.w[sizeof(T) - 2] = q.z;
        p.w[sizeof(T) - 1] = q.w;
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(row + at);
        p.w[0] = q.x;
        p.w[1] = q.y;
      }
    }
  } else {
    Four<T> v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.v[i] = at + 32 * i < n ? row[at + 32 * i] : from_f32<T>(0.f);
    memcpy(&p, &v, sizeof(p));
  }
  return p;
}
__device__ __forceinline__ float value_of(const Words<float>& p, int i) { return __uint_as_float(p.w[i]); }
__device__ __forceinline__ float value_of(const Words<__nv_bfloat16>& p, int i) {
  return __uint_as_float(i & 1 ? p.w[i >> 1] & 0xFFFF0000u : p.w[i >> 1] << 16);
}
__device__ __forceinline__ float value_of(const Words<__half>& p, int i) {
  return __half2float(__ushort_as_half((uint16_t)(i & 1 ? p.w[i >> 1] >> 16 : p.w[i >> 1])));
}

template <bool VEC, typename T>
__device__ __forceinline__ void store4(T* row, int at, int n, const Four<T>& p) {
  if (VEC) {
    if (at < n) *reinterpret_cast<Four<T>*>(row + at) = p;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + 32 * i < n) row[at + 32 * i] = p.v[i];
  }
}

// The sum of a row from its lanes' sums, for all of them.
__device__ __forceinline__ Pair row_sum(float2 hi, float2 lo, Pair* part) {
  const int lane = threadIdx.x & 31, W = blockDim.x >> 5;
  Pair s = add(Pair{hi.x, lo.x}, Pair{hi.y, lo.y});
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Pair t;
    t.hi = __shfl_xor_sync(0xffffffffu, s.hi, o);
    t.lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
    s = add(s, t);
  }
  if (W > 1) {  // one row per CTA then
    if (lane == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = lane < W ? part[lane] : Pair{0.f, 0.f};
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      Pair t;
      t.hi = __shfl_xor_sync(0xffffffffu, s.hi, o);
      t.lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
      s = add(s, t);
    }
    s.hi = __shfl_sync(0xffffffffu, s.hi, 0);
    s.lo = __shfl_sync(0xffffffffu, s.lo, 0);
  }
  return s;
}

// 1 / sqrt(mean + eps) where that is beyond kLeastRoot or kMostRoot, from the row itself: such rows are rare, and read again they cost the
// others no registers.
template <bool VEC, typename T>
__device__ __noinline__ float far_root(const T* row, int at0, int step, int blocks, int n, float eps, Pair s, Pair* part) {
  if (!(mean_of(s, (float)n, eps).hi < 1.f)) {  // (a sum that is no number stays one)
    const Pair m = mean_of(Pair{__fmul_rn(s.hi, 0x1p-100f), __fmul_rn(s.lo, 0x1p-100f)}, (float)n, __fmul_rn(eps, 0x1p-100f));
    return __fmul_rn(recip_root(m), 0x1p-50f);
  }
  // Squares have lost bits, or all of them: once more with the values (below 2^-37 then) times 2^80, of which the smallest number's
  // square still has its 46 bits.
  float2 hi = make_float2(0.f, 0.f), lo = hi;
#pragma unroll 1
  for (int c = 0; c < blocks; ++c) {
    const Words<T> w = load4<VEC>(row, at0 + c * step, n);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 v = __fmul2_rn(make_float2(value_of(w, 2 * i), value_of(w, 2 * i + 1)), make_float2(0x1p80f, 0x1p80f)), p = __fmul2_rn(v, v);
      float2 e;
      two_sum2(hi, p, hi, e);
      lo = __fadd2_rn(lo, __fadd2_rn(e, __ffma2_rn(v, v, make_float2(-p.x, -p.y))));
    }
  }
  if (blockDim.x > 32) __syncthreads();  // the first sum's parts have been read
  const Pair m = mean_of(row_sum(hi, lo, part), (float)n, __fmul_rn(__fmul_rn(eps, 0x1p80f), 0x1p80f));
  return m.hi < 0x1p-96f ? __int_as_float(0x7FC00000) : __fmul_rn(recip_root(m), 0x1p80f);  // beyond float32 below 2^-256
}

// TR: the residual's type, or void.  W warps of a row (blockDim.x / 32), blockDim.y rows per CTA, CH blocks of 128 per warp.  All of a
// row is asked for before anything of it is used; the widest rows, whose values take the registers, four blocks at a time.
template <typename TX, typename TR, int CH, bool VEC>
__global__ void __launch_bounds__(512, CH <= 4 ? 2 : 1) norm_f8_kernel(const NormF8Args a) {
  __shared__ Pair part[16];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, W = blockDim.x >> 5;
  constexpr bool kResid = !std::is_void<TR>::value;
  using TRv = typename std::conditional<kResid, TR, float>::type;
  constexpr int kBatch = CH <= 8 ? CH : 4;
  const int at0 = w * 128 + (VEC ? 4 * lane : lane), step = W * 128;  // of the warp's block c: at0 + c * step
  const int n = a.n;
  Words<TX> in[kBatch];
  Words<TRv> r0[kBatch];
  auto fetch = [&](int row, int c0) {
    const TX* x = static_cast<const TX*>(a.x) + (int64_t)row * a.x_stride;
    const TRv* res = static_cast<const TRv*>(a.resid) + (int64_t)row * a.resid_stride;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      in[j] = load4<VEC>(x, at0 + (c0 + j) * step, n);
      if (kResid) r0[j] = load4<VEC>(res, at0 + (c0 + j) * step, n);
    }
  };
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row < a.n_tok) {  // all warps of a CTA with more than one to a row
    float2 h[CH][2];
    TRv* out = static_cast<TRv*>(a.resid_out) + (int64_t)row * a.resid_out_stride;
#pragma unroll
    for (int c0 = 0; c0 < CH; c0 += kBatch) {
      fetch(row, c0);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        float2(&v)[2] = h[c0 + j];
        v[0] = make_float2(value_of(in[j], 0), value_of(in[j], 1));
        v[1] = make_float2(value_of(in[j], 2), value_of(in[j], 3));
        if constexpr (kResid) {
          Four<TRv> p;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 s = __fadd2_rn(v[i], make_float2(value_of(r0[j], 2 * i), value_of(r0[j], 2 * i + 1)));
            p.v[2 * i] = from_f32<TRv>(s.x);
            p.v[2 * i + 1] = from_f32<TRv>(s.y);
          }
          store4<VEC>(out, at0 + (c0 + j) * step, n, p);
          Words<TRv> back;  // the norm is of what the next block will read
          memcpy(&back, &p, sizeof(back));
          v[0] = make_float2(value_of(back, 0), value_of(back, 1));
          v[1] = make_float2(value_of(back, 2), value_of(back, 3));
        }
      }
    }
    if (a.gamma) {
      float2 hi = make_float2(0.f, 0.f), lo = hi;
      // a square of 12 bits or fewer is a float32
      constexpr bool kExact = sizeof(TRv) == 2 || (!kResid && sizeof(TX) == 2);
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 v = h[c][i], p = __fmul2_rn(v, v);
          float2 e;
          two_sum2(hi, p, hi, e);
          if (!kExact) e = __fadd2_rn(e, __ffma2_rn(v, v, make_float2(-p.x, -p.y)));
          lo = __fadd2_rn(lo, e);
        }
      const Pair s = row_sum(hi, lo, part);
      float r = recip_root(mean_of(s, (float)a.n, a.eps));
      if (__builtin_expect(!(r >= kLeastRoot && r <= kMostRoot), 0)) {
        using TH = typename std::conditional<kResid, TRv, TX>::type;
        const TH* back;
        if constexpr (kResid)
          back = out;
        else
          back = static_cast<const TX*>(a.x) + (int64_t)row * a.x_stride;
        r = far_root<VEC>(back, at0, step, CH, n, a.eps, s, part);
        if constexpr (kBatch < CH)  // the widest rows have no registers to outlive the call (4096 x 28672 in bfloat16: 300 us, 336 if they do)
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const Words<TH> v = load4<VEC>(back, at0 + c * step, n);
            h[c][0] = make_float2(value_of(v, 0), value_of(v, 1));
            h[c][1] = make_float2(value_of(v, 2), value_of(v, 3));
          }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const Words<float> g = load4<VEC>(a.gamma, at0 + c * step, a.n);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          h[c][i] = __fmul2_rn(__fmul2_rn(h[c][i], make_float2(r, r)), make_float2(value_of(g, 2 * i), value_of(g, 2 * i + 1)));
      }
    }
    if (a.y) {
      TX* y = static_cast<TX*>(a.y) + (int64_t)row * a.y_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Four<TX> p;
#pragma unroll
        for (int i = 0; i < 4; ++i) p.v[i] = from_f32<TX>(i & 1 ? h[c][i >> 1].y : h[c][i >> 1].x);
        store4<VEC>(y, at0 + c * step, n, p);
      }
    }
    if (a.q) {
      uint8_t* q = a.q + (int64_t)row * a.q_stride;
      // lane c divides for the warp's block c
      float top = 1.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        // magnitudes compare like their bits, and a NaN above all of them: it is not lost.  (A column from n on is 0, or 0 * r = NaN
        // in a row that is NaN throughout.)
        uint32_t m = 0x0D800000u;  // 2^-100
#pragma unroll
        for (int i = 0; i < 2; ++i)
          m = max(m, max(__float_as_uint(h[c][i].x) & 0x7FFFFFFFu, __float_as_uint(h[c][i].y) & 0x7FFFFFFFu));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == c) top = __uint_as_float(m);
      }
      const float up = __fdiv_rn(448.f, top);
      if (lane < CH && (lane * W + w) * 128 < n) a.scale[(int64_t)(lane * W + w) * a.scale_stride + row] = __fdiv_rn(top, 448.f);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const float t = __shfl_sync(0xffffffffu, up, c);
        const float2 v0 = __fmul2_rn(h[c][0], make_float2(t, t)), v1 = __fmul2_rn(h[c][1], make_float2(t, t));
        const uint32_t codes = (uint32_t)__nv_cvt_float2_to_fp8x2(v0, __NV_SATFINITE, __NV_E4M3) |
                               (uint32_t)__nv_cvt_float2_to_fp8x2(v1, __NV_SATFINITE, __NV_E4M3) << 16;
        Four<uint8_t> p;
        memcpy(&p, &codes, sizeof(p));
        store4<VEC>(q, at0 + c * step, n, p);
      }
    }
  }
}

template <typename TX, typename TR, int CH>
cudaError_t launch_ch(const NormF8Args& a, int warps, int rows, cudaStream_t st) {
  const unsigned grid = (unsigned)((a.n_tok + rows - 1) / rows);
  if (a.vec && a.n % 4 == 0)
    norm_f8_kernel<TX, TR, CH, true><<<grid, dim3(32 * warps, rows), 0, st>>>(a);
  else
    norm_f8_kernel<TX, TR, CH, false><<<grid, dim3(32 * warps, rows), 0, st>>>(a);
  return cudaGetLastError();
}

template <typename TX, typename TR>
cudaError_t launch_t(const NormF8Args& a, cudaStream_t st) {
  const int nb = (a.n + 127) / 128;
  // blocks per warp: few, so that a row is done soon, as long as 16 warps hold it (16411 x 8192: bfloat16 207 us with four, 230 with eight;
  // float32 255 and 263)
  const int ch = nb > 128 ? 16 : nb > 64 ? 8 : 4;
  const int warps = (nb + ch - 1) / ch;
  const int rows = warps == 1 ? 4 : 1;
  if (ch == 16) return launch_ch<TX, TR, 16>(a, warps, rows, st);
  if (ch == 8) return launch_ch<TX, TR, 8>(a, warps, rows, st);
  return launch_ch<TX, TR, 4>(a, warps, rows, st);
}

template <typename TX>
cudaError_t launch_x(const NormF8Args& a, int resid_dtype, cudaStream_t st) {
  if (!a.resid) return launch_t<TX, void>(a, st);
  if (resid_dtype == kTypeF32) return launch_t<TX, float>(a, st);
  return launch_t<TX, TX>(a, st);
}

}  // namespace

cudaError_t launch_norm_f8(const NormF8Args& a, int x_dtype, int resid_dtype, cudaStream_t st) {
  if (x_dtype == kTypeF32) return launch_x<float>(a, resid_dtype, st);
  if (x_dtype == kTypeF16) return launch_x<__half>(a, resid_dtype, st);
  return launch_x<__nv_bfloat16>(a, resid_dtype, st);
}

}  // namespace lrs
