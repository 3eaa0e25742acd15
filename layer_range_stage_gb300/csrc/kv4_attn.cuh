// Device helpers of the attention kernels over the paged 4-bit KV cache.
#pragma once

#include "common.cuh"
#include "kv4.cuh"

namespace lrs {

// x / d for 0 <= x < 2^31, without a division on the device: with 2^(s - 1) < d <= 2^s and m = floor(2^(31 + s) / d) + 1,
// x m / 2^(31 + s) exceeds x / d by less than 1 / d.
struct Quotient {
  int d = 1;
  uint32_t m = 0, shift = 0;
  explicit Quotient(int divisor) : d(divisor) {
    if (d == 1) return;
    int s = 1;
    while ((1ll << s) < d) ++s;
    m = (uint32_t)((1ull << (31 + s)) / (uint32_t)d + 1);
    shift = (uint32_t)(s - 1);
  }
  __device__ __forceinline__ int operator()(int x) const { return d == 1 ? x : (int)(__umulhi((uint32_t)x, m) >> shift); }
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight codes to four half2: h[t] = (code t, code t + 4) - 8, the odd t times 16.  1024 + c is the fp16 number
// 0x6400 | c, and 1024 + 16 c is 0x6400 | c << 4: one logic operation and one addition per pair, both exact.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}
// The exponent's bits in a register that the compiler takes for a variable: as a constant they would make two
// operations of and_or, which has room for one immediate.
__device__ __forceinline__ uint32_t exponent_bits() {
  uint32_t y;
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(y));
  return y;
}
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t ex, uint32_t (&h)[4]) {
  const __half2 o1 = __floats2half2_rn(-1032.f, -1032.f), o16 = __floats2half2_rn(-1152.f, -1152.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = i ? w >> 8 : w;
    const uint32_t a = and_or(x, 0x000f000fu, ex), b = and_or(x, 0x00f000f0u, ex);
    const __half2 ha = __hadd2(*reinterpret_cast<const __half2*>(&a), o1);
    const __half2 hb = __hadd2(*reinterpret_cast<const __half2*>(&b), o16);
    h[2 * i] = *reinterpret_cast<const uint32_t*>(&ha);
    h[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&hb);
  }
}

__device__ __forceinline__ float2 h2_to_f2(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t x, y, d;
  float2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t x, y, d;
  float2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z, d;
  float2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

// The largest of a, |b| and |c|; NaN loses.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return y;
}

__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight neighbouring elements (i a multiple of 8, rows 16-byte aligned).
__device__ __forceinline__ void load8(const void* p, int dtype, long long i, float (&v)[8]) {
  if (dtype == KV4_F32) {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const float4 x = q[0], y = q[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    return;
  }
  const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (dtype == KV4_F16) {
      const float2 f = h2_to_f2(w[k]);
      v[2 * k] = f.x, v[2 * k + 1] = f.y;
    } else {
      v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void store_elem(void* p, int dtype, long long i, float v) {
  if (dtype == KV4_F32) reinterpret_cast<float*>(p)[i] = v;
  else if (dtype == KV4_F16) reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
  else reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ int seq_positions(const Kv4AttnArgs& a, int s) {
  const long long most = min((long long)a.max_len, (long long)a.table_stride * a.c.page_len);
  return (int)max(0ll, min((long long)a.seq_len[s], most));
}
// Query tokens of a sequence that get an output, and the first.
__device__ __forceinline__ int seq_tokens(const Kv4AttnArgs& a, int s, int* start) {
  const int b = a.cu_q[s], e = a.cu_q[s + 1];
  *start = b;
  if (b < 0 || e <= b || e > a.n_tok) return 0;
  return e - b;
}

}  // namespace lrs
