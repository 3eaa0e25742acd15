// Attention over the paged 4-bit KV cache (sm_103a).
//
// Mathematics.  With a score's exponent in base 2, z_j = log2(e) / sqrt(D) * sum_b sk_jb sum_{d in b} q_d (c_jd - 8),
//   o_d = sum_j 2^(z_j - r) sv_jb (c'_jd - 8) / sum_j 2^(z_j - r)
// for any r.  The codes minus 8 are exact in fp16, so both inner products run on the tensor cores
// (mma.sync m16n8k16, float32 accumulation) on integers; the block scales multiply the K product's partial
// sums and, because V's position is the summed index, the probabilities: x_jb = 2^(z_j - r) sv_jb.
// q (scaled by a power of two into fp16's range) and x are each split into a high and a low fp16 value, 22
// bits together: the result is float32's, not fp16's.  r runs above max_j (z_j + log2 |sv_j|) - 11, so that the
// largest x lies near 2^11 .. 2^15 whatever the scales are, and fp16's range ends 2^36 below it.
//
// Split of the work.  Rows (sequence, KV head, block of columns) times units of 128 positions form one line
// of units in memory order, cut into equal pieces, one per resident CTA: ragged batches load every SM
// alike, whatever the lengths, which only the device knows.  A row has kRowCost empty units more, at its front, for what
// a row costs by itself (its q, the merge of the warps, its output).  A row cut by piece borders is merged by the last
// of its CTAs to arrive, in the order of the positions.
//
// What bounds it: instructions, not bytes.  A tile of 16 positions is 2304 bytes and 496 instructions of a warp (unpacking
// 4096 codes alone takes 130), which the four schedulers of an SM issue at about three quarters of their rate.  One token on
// 131001 positions (32/8 heads of 128): 56 us for 151 MB, 2.7 TB/s; 64 ragged sequences of 128 .. 4096: 66 us for 166 MB; up
// to 5 drafts of 16 sequences: 27 us, where every eight columns read the cache again.  Two tiles a round, for more
// independent work, spilled and took 58, 68 and 30 us.

#include <atomic>
#include <cfloat>

#include "common.cuh"
#include "kernels.cuh"
#include "kv4_attn.cuh"

namespace lrs {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kUnitTiles = kWarps;  // a unit: one tile of 16 positions per warp
constexpr int kStages = 4;          // tiles in flight per warp, less one
constexpr int kFlush = 16;          // tiles between two flushes of the accumulators
constexpr int kMaxCtas = kKv4MaxCtas;
constexpr int kRowCost = 4;  // 64 ragged sequences (64/8 heads): 91 us with 0, 74 with 2, 68 with 3, 69 with 5
constexpr int kSlack = 4;           // r is raised when a score passes it by 2^kSlack
constexpr float kTop = 11.f;

// floats of a partial result in the workspace: eight columns' outputs, (r, sum) of each column
__host__ __device__ constexpr int slot_floats(int D) { return 8 * D + 16; }

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Units of a row of this many positions, the empty ones among them.
__device__ __forceinline__ int row_units(int len) {
  return kRowCost + max(1, (len + kUnitTiles * kKv4Tile - 1) / (kUnitTiles * kKv4Tile));
}
// Quotients of counts, which rarely need 64 bits.
__device__ __forceinline__ long long quotient(long long x, int y) {
  return x >> 32 ? x / y : (long long)((uint32_t)x / (uint32_t)y);
}

// A segment: units [begin, end) of the row (sequence, KV head, block of columns) that has [unit, unit + units).
struct AttnRow {
  int head, cbase, ncols;    // KV head, first column, columns of the sequence
  int start, count, len;     // first query token of the sequence, its tokens, its positions
  int units;
  long long unit, begin, end;
};

template <int D, int NC>
struct __align__(16) AttnSmem {
  uint8_t ring[kWarps][kStages][kv4_tile_bytes(D)];
  float acc[kWarps][8 * D];     // flushed accumulators, then the warps' results: [register][lane]
  float ref[kWarps][8], sum[kWarps][8];
  long long wsum[kWarps];
  long long first_unit;         // of the sequence that holds this CTA's first unit
  long long piece, longer;      // piece c of the line begins at unit c * piece + min(c, longer)
  AttnRow seg;                  // the segment in work
  int first_seq;
  int last, part0, parts;
};

// Columns: NC = 8 has eight (token, head of the group) pairs, their high parts in rows 0-7 and their low parts in
// rows 8-15 of the score product, and two products for V.  NC = 4 has four: rows 4-7 repeat rows 0-3, and the
// columns 4-7 of the V product carry the low parts, so one product does.
template <int D, int NC>
__global__ void __launch_bounds__(kThreads, 2) kv4_attn_kernel(const Kv4AttnArgs a, int dtype, unsigned* counters, float* slots, const Quotient by_group,
                    const Quotient by_page) {
  constexpr int NB = D / 32, MT = D / 16;  // blocks of a row, row tiles of the V product
  constexpr int TILE = kv4_tile_bytes(D), HALF = kv4_half(D), CODES = kv4_codes(D);
  extern __shared__ __align__(16) unsigned char smem_raw[];
  AttnSmem<D, NC>& sm = *reinterpret_cast<AttnSmem<D, NC>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, tig = lane & 3;
  const int group = by_group.d, tpp = by_page.d;  // query heads per KV head, tiles per page

  // ---- this CTA's piece of the line of units
  const int cta = blockIdx.x;
  long long u, u_end;
  {
    long long total = 0;
    const int per = (a.n_seqs + kThreads - 1) / kThreads;
    const int s0 = min(a.n_seqs, tid * per), s1 = min(a.n_seqs, s0 + per);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
      int start;
      const int c = min(seq_tokens(a, s, &start), a.max_q);
      const int units = row_units(seq_positions(a, s));
      mine += (long long)((c * (long long)group + NC - 1) / NC) * a.c.n_kv_heads * units;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) sm.wsum[warp] = incl;
    if (tid == 0) sm.first_seq = a.n_seqs;
    __syncthreads();
    long long before = incl - mine;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.wsum[w];
      total += sm.wsum[w];
    }
    const int ncta = (int)min((long long)gridDim.x, total);  // every piece has a unit
    if (cta >= ncta) return;
    const long long piece = total / ncta, longer = total % ncta;
    u = cta * piece + min((long long)cta, longer);
    u_end = u + piece + (cta < longer ? 1 : 0);
    if (tid == 0) {
      sm.piece = piece;
      sm.longer = longer;
    }
    if (u >= before && u < before + mine) {
      long long at = before;
      for (int s = s0; s < s1; ++s) {
        int start;
        const int c = min(seq_tokens(a, s, &start), a.max_q);
        const int units = row_units(seq_positions(a, s));
        const long long n = (long long)((c * (long long)group + NC - 1) / NC) * a.c.n_kv_heads * units;
        if (u < at + n) {
          sm.first_seq = s;
          sm.first_unit = at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
  }
  int seq = sm.first_seq;
  long long seq_unit = sm.first_unit;

  float acc[MT][4];
  float ref = -INFINITY;               // of column gid
  float2 sum = make_float2(0.f, 0.f);  // over this lane's positions, the first and the second of each pair
  float ref_flushed = -INFINITY;
  bool flushed = false, pending = false;  // pending: a segment's sums wait to be put down
  float* my_acc = sm.acc[warp];

  // Each round finds the next segment and starts its copies, puts the last one's results down meanwhile, and runs
  // the next one.
  while (true) {
    AttnRow row = {};
    int n_it = 0, t_begin = 0, lim_lo = 0;
    bool more = u < u_end;
    uint32_t present = 0;            // bit i % 32: tile i is there
    int page_ids = -1, in_page = 0;  // of tile number 32 * batch + lane
    const int* trow = nullptr;
    auto issue = [&](int i) {
      if (i < n_it) {
        if ((i & 31) == 0) {
          const int t = t_begin + warp + (i + lane) * kWarps;
          const int pg = by_page(t);
          in_page = t - pg * tpp;
          page_ids = i + lane < n_it ? trow[pg] : -1;
          if (page_ids < 0 || page_ids >= a.c.n_pages) page_ids = -1;
        }
        const int id = __shfl_sync(0xffffffffu, page_ids, i & 31), in = __shfl_sync(0xffffffffu, in_page, i & 31);
        if (id >= 0) {
          present |= 1u << (i & 31);
          const uint8_t* src = a.c.data + (((long long)id * a.c.n_kv_heads + row.head) * tpp + in) * TILE;
          uint8_t* dst = sm.ring[warp][i % kStages];
#pragma unroll
          for (int j = 0; j < (TILE / 16 + 31) / 32; ++j) {
            const int o = lane + 32 * j;
            if (o < TILE / 16) cp_async16(dst + o * 16, src + o * 16);
          }
        } else {
          present &= ~(1u << (i & 31));
        }
      }
      cp_async_commit();
    };
    if (more) {
      while (true) {
        row.count = seq_tokens(a, seq, &row.start);
        row.len = seq_positions(a, seq);
        row.ncols = min(row.count, a.max_q) * group;
        row.units = row_units(row.len);
        const int cblocks = (row.ncols + NC - 1) / NC;
        const long long all = (long long)cblocks * a.c.n_kv_heads * row.units;
        if (u < seq_unit + all) {
          const long long r = quotient(u - seq_unit, row.units);
          row.unit = seq_unit + r * row.units;
          row.head = (int)quotient(r, cblocks);
          row.cbase = (int)(r - (long long)row.head * cblocks) * NC;
          break;
        }
        seq_unit += all;  // the next sequence (those without a token have no unit)
        ++seq;
      }
      // from here on the row's own units alone
      row.unit += kRowCost;
      row.units -= kRowCost;
      row.begin = max(u, row.unit);
      row.end = min(u_end, row.unit + row.units);
      more = row.begin < row.end;  // the piece may end among the empty ones
    }
    if (more) {
      u = row.end;
      t_begin = (int)(row.begin - row.unit) * kUnitTiles;
      const int k_hi = by_group(min(row.ncols - 1, row.cbase + NC - 1)), k_lo = by_group(row.cbase);
      const int lim_hi = max(0, row.len - row.count + k_hi + 1);  // positions that some column sees
      lim_lo = max(0, row.len - row.count + k_lo + 1);            // positions that every column sees
      const int t_end = min((int)(row.end - row.unit) * kUnitTiles, (lim_hi + kKv4Tile - 1) / kKv4Tile);
      // the warp's tiles: t_begin + warp, + kWarps, ...
      n_it = max(0, (t_end - t_begin - warp + kWarps - 1) / kWarps);
      trow = a.table + (long long)seq * a.table_stride;
      // the segment's q into L1 (a line per lane), while its pages are looked up and the last segment's results put down
      const int col = row.cbase + (lane >> 2), esize = dtype == KV4_F32 ? 4 : 2;
      if ((lane >> 2) < NC && col < row.ncols && (lane & 3) * 128 < D * esize) {
        const int k = by_group(col);
        const long long at = (long long)(row.start + k) * a.q_stride + (row.head * group + col - k * group) * D;
        uint32_t unused;
        asm volatile("ld.global.ca.b32 %0, [%1];" : "=r"(unused) : "l"((const char*)a.q + at * esize + (lane & 3) * 128));
      }
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) issue(i);
    }
    if (pending) {
      // ---- the warp's result
      float den = sum.x + sum.y;
      den += __shfl_xor_sync(0xffffffffu, den, 1);
      den += __shfl_xor_sync(0xffffffffu, den, 2);
      {
        const float keep = flushed ? (ref_flushed == ref ? 1.f : exp2_approx(ref_flushed - ref)) : 0.f;
        const float k0 = __shfl_sync(0xffffffffu, keep, 8 * tig), k1 = __shfl_sync(0xffffffffu, keep, 8 * tig + 4);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float* f = my_acc + (4 * m + j) * 32 + lane;
            float v = flushed ? fmaf(*f, j & 1 ? k1 : k0, acc[m][j]) : acc[m][j];
            if (j >= 2) v *= 0.0625f;  // the odd dims' codes were times 16
            if constexpr (NC == 4) v += __shfl_xor_sync(0xffffffffu, v, 2);  // high and low part
            *f = v;
          }
      }
      if (tig == 0) {
        sm.ref[warp][gid] = ref;
        sm.sum[warp][gid] = den;
      }
      __syncthreads();

      const AttnRow& done = sm.seg;
      // ---- the CTA's result: entry e = register * 32 + lane holds (dim, column)
      const bool split = done.begin > done.unit || done.end < done.unit + done.units;
      float* slot = nullptr;
      if (split) slot = slots + (size_t)(2 * cta + (done.begin == done.unit ? 1 : 0)) * slot_floats(D);
      auto entry_col = [&](int e) { return (e & 3) * 2 + ((e >> 5) & 1); };
      // Output of column c (of the block): its row, and a value at entry e.
      auto out_row = [&](int c) {
        const int at = done.cbase + c, k = by_group(at);
        return (long long)(done.start + k) * a.out_stride + (done.head * group + at - k * group) * D;
      };
      auto put = [&](long long row_at, int e, float v) {
        store_elem(a.out, dtype, row_at + (e >> 8) * 32 + ((e & 31) >> 2) * 4 + ((e >> 7) & 1) * 2 + ((e >> 6) & 1), v);
      };
      {
        static_assert(kThreads % 256 == 0, "all entries of a thread have one column");
        const int c = entry_col(tid);
        float top = -INFINITY, s = 0.f, k[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, k[w] = sm.ref[w][c]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          k[w] = k[w] == top ? 1.f : exp2_approx(k[w] - top);  // 0 for a warp without a position; NaN sums stay NaN
          s = fmaf(sm.sum[w][c], k[w], s);
        }
        const bool real = !split && c < NC && done.cbase + c < done.ncols;
        const long long row_at = real ? out_row(c) : 0;
        const float inv = s != 0.f ? 1.f / s : 0.f;
        for (int e = tid; e < 8 * D; e += kThreads) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v = fmaf(sm.acc[w][e], k[w], v);
          if (split) __stcg(slot + e, v);
          else if (real) put(row_at, e, s != 0.f ? v * inv : 0.f);
        }
        if (split && tid < 64 && (tid >> 2 & 7) == 0) {  // registers 0 and 1 of lanes 0-3: one thread for every column
          __stcg(slot + 8 * D + c, top);
          __stcg(slot + 8 * D + 8 + c, s);
        }
      }
      if (split) {
        __syncthreads();
        if (tid == 0) {
          const long long piece = sm.piece, cut = sm.longer * (piece + 1);
          auto owner = [&](long long x) {  // of unit x
            return (int)(x < cut ? x / (piece + 1) : sm.longer + (x - cut) / piece);
          };
          const int c0 = owner(done.unit), parts = owner(done.unit + done.units - 1) - c0 + 1;
          const unsigned old = atom_add_acq_rel(&counters[c0], 1u);
          sm.last = old == (unsigned)(parts - 1);
          if (sm.last) counters[c0] = 0;
          sm.part0 = c0;
          sm.parts = parts;
        }
        __syncthreads();
        if (sm.last) {
          const int c0 = sm.part0, parts = sm.parts;
          // weights of the parts, then the sums in the order of the positions
          float* wt = &sm.acc[0][0];  // [part][8]: r, then the weight
          float* den = &sm.sum[0][0];
          auto part = [&](int i) { return slots + (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * slot_floats(D); };
          for (int i = tid; i < parts * 8; i += kThreads) wt[i] = __ldcg(part(i >> 3) + 8 * D + (i & 7));
          __syncthreads();
          // a warp per column
          {
            float top = -INFINITY, s = 0.f;
            for (int i = lane; i < parts; i += 32) top = fmaxf(top, wt[i * 8 + warp]);
            top = warp_max(top);
            for (int i = lane; i < parts; i += 32) {
              const float r_i = wt[i * 8 + warp];
              const float k = r_i == top ? 1.f : exp2_approx(r_i - top);
              wt[i * 8 + warp] = k;
              s = fmaf(__ldcg(part(i) + 8 * D + 8 + warp), k, s);
            }
            s = warp_sum(s);
            if (lane == 0) den[warp] = s;
          }
          __syncthreads();
          for (int e4 = tid; e4 < 2 * D; e4 += kThreads) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 16
            for (int i = 0; i < parts; ++i) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(part(i)) + e4);
              const float* w = wt + i * 8;
              const int b = (e4 >> 3) & 1;
              v[0] = fmaf(x.x, w[b], v[0]);
              v[1] = fmaf(x.y, w[2 + b], v[1]);
              v[2] = fmaf(x.z, w[4 + b], v[2]);
              v[3] = fmaf(x.w, w[6 + b], v[3]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int c = entry_col(4 * e4 + j);
              if (c < NC && done.cbase + c < done.ncols) put(out_row(c), 4 * e4 + j, den[c] != 0.f ? v[j] / den[c] : 0.f);
            }
          }
        }
      }
      __syncthreads();
    }
    if (!more) break;
    if (tid == 0) sm.seg = row;  // read after the barriers that follow the segment's tiles

    // ---- the columns' q as the A operand: rows gid (high) and gid + 8 (low)
    const int col = row.cbase + (NC == 8 ? gid : gid & 3);
    const bool col_live = col < row.ncols;
    const int col_k = by_group(col);
    const int lim = col_live ? max(0, row.len - row.count + col_k + 1) : 0;
    uint32_t qa[2 * NB][4];
    float zscale;
    {
      const long long base = col_live ? (long long)(row.start + col_k) * a.q_stride + (row.head * group + col - col_k * group) * D : 0;
      float qv[NB][8], top = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (col_live) {
          load8(a.q, dtype, base + b * 32 + tig * 8, qv[b]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) qv[b][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(qv[b][i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the largest |q| to 2^13 .. 2^14 by a power of two (2^-100 is as good as 0)
      const int e = top <= FLT_MAX ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 0;
      zscale = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(e - 13 + 127) << 23);
      const float up[2] = {__uint_as_float((uint32_t)(13 - e + 127) << 23), __uint_as_float((uint32_t)(9 - e + 127) << 23)};
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int o = 0; o < 2; ++o) {  // dims 2 s + o and 2 s + o + 4 of the lane's eight; odd ones face codes times 16
            const float2 x = mul2(make_float2(qv[b][2 * s + o], qv[b][2 * s + o + 4]), make_float2(up[o], up[o]));
            const __half2 h = __floats2half2_rn(x.x, x.y);
            const float2 l = fma2(__half22float2(h), make_float2(-1.f, -1.f), x);
            const __half2 r = __floats2half2_rn(l.x, l.y);
            qa[2 * b + s][2 * o] = *reinterpret_cast<const uint32_t*>(&h);
            qa[2 * b + s][2 * o + 1] = *reinterpret_cast<const uint32_t*>(&r);
          }
    }

#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
    ref = ref_flushed = -INFINITY;
    sum = make_float2(0.f, 0.f);
    flushed = false;
    const uint32_t ex = exponent_bits();
    int since = 0;
    for (int i = 0; i < n_it; ++i) {
      cp_async_wait_group<kStages - 2>();
      __syncwarp();
      const bool here = present >> (i & 31) & 1;
      issue(i + kStages - 1);
      if (!here) continue;
      const uint8_t* tile = sm.ring[warp][i % kStages];
      const int pos0 = (t_begin + warp + i * kWarps) * kKv4Tile;

      // scores of positions 8 n + 2 tig + {0, 1} and column gid
      float2 z[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint32_t kw[NB], ks[NB];  // ks: fp16 pairs (blocks 2 i, 2 i + 1) of the first, then of the second position
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(tile + (8 * n + gid) * (D / 2) + tig * 16);
          kw[0] = w.x, kw[1] = w.y, kw[2] = w.z, kw[3] = w.w;
          const uint4 s = *reinterpret_cast<const uint4*>(tile + CODES + (8 * n + 2 * tig) * (2 * NB));
          ks[0] = s.x, ks[1] = s.y, ks[2] = s.z, ks[3] = s.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(tile + (8 * n + gid) * (D / 2) + tig * 8);
          kw[0] = w.x, kw[1] = w.y;
          const uint2 s = *reinterpret_cast<const uint2*>(tile + CODES + (8 * n + 2 * tig) * (2 * NB));
          ks[0] = s.x, ks[1] = s.y;
        }
        z[n] = make_float2(0.f, 0.f);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t h[4];
          codes_to_half(kw[b], ex, h);
          const float zero[4] = {0.f, 0.f, 0.f, 0.f};
          float c[4];
          mma16816(c, qa[2 * b], h[0], h[1], zero);
          mma16816(c, qa[2 * b + 1], h[2], h[3], c);
          const float2 sa = h2_to_f2(ks[b / 2]), sb = h2_to_f2(ks[NB / 2 + b / 2]);
          const float2 both = add2(make_float2(c[0], c[1]), make_float2(c[2], c[3]));  // high and low part of q
          z[n] = fma2(b & 1 ? make_float2(sa.y, sb.y) : make_float2(sa.x, sb.x), both, z[n]);
        }
      }

      // V's scales, (first, second position) of each block; those of positions that the column does not see count as 0
      float2 vs[2][NB];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint32_t s[NB];
        if constexpr (D == 128) {
          const uint4 u4 = *reinterpret_cast<const uint4*>(tile + HALF + CODES + (8 * n + 2 * tig) * (2 * NB));
          s[0] = u4.x, s[1] = u4.y, s[2] = u4.z, s[3] = u4.w;
        } else {
          const uint2 u2 = *reinterpret_cast<const uint2*>(tile + HALF + CODES + (8 * n + 2 * tig) * (2 * NB));
          s[0] = u2.x, s[1] = u2.y;
        }
#pragma unroll
        for (int b = 0; b < NB / 2; ++b) {
          const float2 first = h2_to_f2(s[b]), second = h2_to_f2(s[NB / 2 + b]);
          vs[n][2 * b] = make_float2(first.x, second.x);
          vs[n][2 * b + 1] = make_float2(first.y, second.y);
        }
      }
      // An infinite scale of K counts as NaN: a score of -infinity would drop its position without a word
#pragma unroll
      for (int n = 0; n < 2; ++n) z[n] = fma2(z[n], make_float2(0.f, 0.f), z[n]);
      if (pos0 + kKv4Tile > lim_lo) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int at = pos0 + 8 * n + 2 * tig;
          if (at >= lim) z[n].x = -INFINITY;
          if (at + 1 >= lim) z[n].y = -INFINITY;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if (at >= lim) vs[n][b].x = 0.f;
            if (at + 1 >= lim) vs[n][b].y = 0.f;
          }
        }
      }
      // the largest z + log2 of a position's largest scale (at least fp16's smallest; NaN loses; an infinity counts as fp16's
      // largest, so that it makes its own block NaN, through its product, and nothing of the others)
      float most = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float2 top = make_float2(5.9604645e-8f, 5.9604645e-8f);
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
          top.x = max_abs(top.x, vs[n][b].x, vs[n][b + 1].x);
          top.y = max_abs(top.y, vs[n][b].y, vs[n][b + 1].y);
        }
        most = fmaxf(most, fmaf(z[n].x, zscale, log2_approx(fminf(top.x, 65504.f))));
        most = fmaxf(most, fmaf(z[n].y, zscale, log2_approx(fminf(top.y, 65504.f))));
      }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const bool raise = most - kTop > ref + kSlack;
      if (__any_sync(0xffffffffu, raise)) {
        const float now = raise ? most - kTop : ref;
        const float keep = ref == now ? 1.f : exp2_approx(ref - now);
        ref = now;
        sum = mul2(sum, make_float2(keep, keep));
        const float k0 = __shfl_sync(0xffffffffu, keep, 8 * tig), k1 = __shfl_sync(0xffffffffu, keep, 8 * tig + 4);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[m][0] *= k0;
          acc[m][1] *= k1;
          acc[m][2] *= k0;
          acc[m][3] *= k1;
        }
      }
      const float base = ref == -INFINITY ? 0.f : ref;
      float2 p[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        p[n].x = exp2_approx(fmaf(z[n].x, zscale, -base));
        p[n].y = exp2_approx(fmaf(z[n].y, zscale, -base));
        sum = add2(sum, p[n]);
      }

      // x = p * scale, split; then the product with V's codes
      uint32_t vw[2][NB];  // [half][block]: the lane's four dims of the first position, then of the second
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(tile + HALF + n * 4 * D + lane * 16);
          vw[n][0] = __byte_perm(w.x, w.z, 0x5410), vw[n][1] = __byte_perm(w.x, w.z, 0x7632);
          vw[n][2] = __byte_perm(w.y, w.w, 0x5410), vw[n][3] = __byte_perm(w.y, w.w, 0x7632);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(tile + HALF + n * 4 * D + lane * 8);
          vw[n][0] = __byte_perm(w.x, w.y, 0x5410), vw[n][1] = __byte_perm(w.x, w.y, 0x7632);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float2 x = mul2(p[n], vs[n][b]);
          const __half2 h = __floats2half2_rn(x.x, x.y);
          const float2 f = __half22float2(h);
          const float2 rest = fma2(f, make_float2(-1.f, -1.f), x);
          const __half2 l = __floats2half2_rn(rest.x, rest.y);
          hi[n] = *reinterpret_cast<const uint32_t*>(&h);
          lo[n] = *reinterpret_cast<const uint32_t*>(&l);
        }
        uint32_t v0[4], v1[4];
        codes_to_half(vw[0][b], ex, v0);  // dims 4 gid + {0, 1, 2, 3} of the block; (first, second position)
        codes_to_half(vw[1][b], ex, v1);
        const uint32_t even[4] = {v0[0], v0[1], v1[0], v1[1]}, odd[4] = {v0[2], v0[3], v1[2], v1[3]};
        if constexpr (NC == 8) {
          mma16816(acc[2 * b], even, hi[0], hi[1], acc[2 * b]);
          mma16816(acc[2 * b + 1], odd, hi[0], hi[1], acc[2 * b + 1]);
          mma16816(acc[2 * b], even, lo[0], lo[1], acc[2 * b]);
          mma16816(acc[2 * b + 1], odd, lo[0], lo[1], acc[2 * b + 1]);
        } else {
          const uint32_t x0 = gid < 4 ? hi[0] : lo[0], x1 = gid < 4 ? hi[1] : lo[1];
          mma16816(acc[2 * b], even, x0, x1, acc[2 * b]);
          mma16816(acc[2 * b + 1], odd, x0, x1, acc[2 * b + 1]);
        }
      }
      // the tensor cores' additions truncate: their chains stay short, longer sums are rounded to nearest
      if (++since == kFlush) {
        since = 0;
        const float keep = flushed ? (ref_flushed == ref ? 1.f : exp2_approx(ref_flushed - ref)) : 0.f;
        const float k0 = __shfl_sync(0xffffffffu, keep, 8 * tig), k1 = __shfl_sync(0xffffffffu, keep, 8 * tig + 4);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float* f = my_acc + (4 * m + j) * 32 + lane;
            *f = flushed ? fmaf(*f, j & 1 ? k1 : k0, acc[m][j]) : acc[m][j];
            acc[m][j] = 0.f;
          }
        ref_flushed = ref;
        flushed = true;
      }
    }
    pending = true;
  }
}

template <int D, int NC>
cudaError_t launch(const Kv4AttnArgs& a, int dtype, cudaStream_t st) {
  constexpr size_t smem = sizeof(AttnSmem<D, NC>);
  static_assert(kWarps == 8, "a warp per column");
  static_assert(smem <= 113 * 1024, "two CTAs share an SM");
  static_assert(sizeof(((AttnSmem<D, NC>*)nullptr)->acc) >= kMaxCtas * 8 * sizeof(float), "weights of a row's parts");
  auto* kern = kv4_attn_kernel<D, NC>;
  static std::atomic<uint64_t> ready{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  // no more CTAs than units at the stated bounds
  const int group = a.n_q_heads / a.c.n_kv_heads;
  const long long len = min((long long)a.max_len, (long long)a.table_stride * a.c.page_len);
  const long long most = (long long)a.n_seqs * a.c.n_kv_heads * (((long long)a.max_q * group + NC - 1) / NC) *
                         ((len + kUnitTiles * kKv4Tile - 1) / (kUnitTiles * kKv4Tile));
  const int grid = (int)min(min(most, 2ll * sm_count()), (long long)kMaxCtas);
  unsigned* counters = (unsigned*)a.ws;
  kern<<<grid, kThreads, smem, st>>>(a, dtype, counters, (float*)((char*)a.ws + kKv4CounterBytes), Quotient(group),
                                     Quotient(a.c.page_len / kKv4Tile));
  return cudaGetLastError();
}

}  // namespace

// Few columns (query tokens of a sequence times heads of a group) run on the kernel above, which reads the cache again for
// every eight of them; many on the tiles of kernels_kv4_chunk.cu.  Measured (us), with z = n_seqs * n_kv_heads * max_len in
// millions: here 12 + `few` z per eight columns; there about 20 + `many` z per 128 rows, STAGE_BF16 per 256.  16 sequences of 4096 with
// 8 KV heads (z = 0.52), head_dim 128, float32, float16, bfloat16: 32 columns 99 here and 111, 82, 76 there, 64 columns 185
// and the same; head_dim 64: 32 columns 64 and 93, 78, 70, 64 columns 117 and the same.  4 of 512 (z = 0.016), head_dim 128: 64
// columns 20 and 23, 21, 21, 256 columns 43 and 23, 21, 27.
constexpr int kFewColumns = 24;

bool kv4_many_columns(const Kv4AttnArgs& a, int head_dim, int dtype) {
  const long long cols = (long long)a.max_q * (a.n_q_heads / a.c.n_kv_heads);
  if (cols <= kFewColumns) return false;
  // Bounds so loose that looking through the row tiles alone would take a tenth of a second
  if ((cols + 127) / 128 * a.c.n_kv_heads * a.n_seqs > kKv4ChunkItems) return false;
  const double z = 1e-6 * a.n_seqs * a.c.n_kv_heads * a.max_len;
  const bool wide = head_dim == 128;
  const double few = wide ? 43. : 25.;
  const double many = dtype == KV4_F32 ? (wide ? 175. : 139.) : dtype == KV4_F16 ? (wide ? 118. : 111.) : (wide ? 155. : 126.);
  const int rows = dtype == KV4_BF16 ? 256 : 128;
  return (few * ((cols + 7) / 8) - many * ((cols + rows - 1) / rows)) * z > 8.;
}

size_t kv4_attention_ws_bytes(int, int n_q_heads, int n_kv_heads, int head_dim, int max_q, int) {
  const size_t few = kKv4CounterBytes + (size_t)2 * kMaxCtas * slot_floats(head_dim) * sizeof(float);
  return (long long)max_q * (n_q_heads / n_kv_heads) > kFewColumns ? max(few, kv4_chunk_ws_bytes(head_dim)) : few;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int head_dim, int dtype, cudaStream_t st) {
  if (kv4_many_columns(a, head_dim, dtype)) return launch_kv4_chunk(a, head_dim, dtype, st);
  const long long cols = (long long)a.max_q * (a.n_q_heads / a.c.n_kv_heads);
  if (head_dim == 128) return cols <= 4 ? launch<128, 4>(a, dtype, st) : launch<128, 8>(a, dtype, st);
  return cols <= 4 ? launch<64, 4>(a, dtype, st) : launch<64, 8>(a, dtype, st);
}

}  // namespace lrs
