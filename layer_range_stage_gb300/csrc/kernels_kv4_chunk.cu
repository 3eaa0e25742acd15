// Attention of many query tokens per sequence (prompt chunks) over the paged 4-bit KV cache (sm_103a): tcgen05 tiles.
//
// A work item is 128 rows -- (token, head of the group) pairs of one sequence and KV head -- against the positions they
// see, in tiles of 64.  One CTA per SM goes through its items (the longest first, dealt forth and back) without a barrier
// between them: a tile's number n runs on over the items, and the copies and the expansion of the next item's first
// tiles go on while the last item's results are put down.  Roles, joined by mbarriers:
//   warps 0-7   softmax: warp w has the rows 32 (w % 4) .. + 31 (the TMEM lanes it may read), w / 4 the half of a tile's
//               positions, and of the output's dims, that its threads take;
//   warps 8-15  turn the packed tiles into fp16 operands in the tensor core's swizzled layout, K as [position][dim],
//               V as [dim][position]: four warps have the even tiles, four the odd ones, so each has two tiles' time
//               for its chain of waits, reads and writes;
//   warp 16     issues the products: S = Q K^T and O = P V, with Q and P read from TMEM (an operand of 128 rows from shared
//               memory would be read again by every product);
//   warp 17     copies the packed tiles in (bulk copies, up to four tiles ahead).
// What bounds it: the latency of a tile's chain (scores, softmax, probabilities, outputs) and of an item's ends (its q, its
// results); the tensor cores are busy for 25 % of the time (4 x 512 rows of 32/8 heads, STAGE_F32: 57 us) and 34 % (2 x 1024
// rows on 8192 positions, STAGE_BF16, the second kernel below: 342 us, 682 TFLOP/s), the schedulers for 41 and 48 %.
// The tensor cores' additions truncate: over a long sum the result shrinks (by 6e-7 of itself per tile of 64 positions, 15 %
// over 16 million).  So in STAGE_F32 every tile's O is added to float32 registers, rounded to nearest, and the products with
// low parts come first, where the sums they truncate are still small: 2e-6 of error became 5e-7.  The 16-bit types keep
// the sum in TMEM, where a row's change of reference, which is rare, rescales it, for a chain of kChain tiles (7e-5 of the
// sum); then it is added to float32 sums in the workspace and begins again.
//
// Precision: a value s (c - 8) has 15 significant bits, so two fp16 numbers hold it exactly; q and the probabilities are
// float32 and two fp16 numbers hold 22 bits.  STAGE_F32 multiplies high by high, low by high and high by low (three
// products each for S and O); STAGE_F16 has an exact q in one number and keeps K and V exact (two); STAGE_BF16, whose
// output keeps 8 bits, rounds K, V and the probabilities to fp16 once (one).
// Values of K are multiples of 2^-24 and, with scales below 4096, at most 2^15: fp16's range holds them as they are (a
// subnormal one exactly, in one number).  In the rare tile with a scale from 4096 on (rows of 32768), each position
// has a power of its own, 1 where its own scales are below, which its score is multiplied by: what other positions hold,
// those that a row does not see among them, changes nothing, and the position's own values lose 2^-33 of its largest.
// V's scales are multiplied by a power of two that brings the largest to 2^10 .. 2^12, and the probabilities by its inverse: so
// the largest p_j |v_j| of a row, whatever the scales, has a probability near fp16's top, and what lies
// 2^27 (STAGE_F32: 2^34) or more below it is lost.  Multiplied by powers of two up (from scales below 4096), multiples of 2^-24
// stay what they are, so values of V are exact like K's.  In STAGE_F32 each position has its power.  In the 16-bit types a tile's
// positions share one where their largest scales lie within a factor of 16, which rows of a model mostly do and which saves
// a multiplication and an addition per score; in other tiles each has its own.

#include <atomic>
#include <cfloat>
#include <climits>
#include <cstddef>

#include "kernels.cuh"
#include "kv4_attn.cuh"
#include "tc.cuh"

namespace lrs {

namespace {

constexpr int kRowsTile = 128, kPosTile = 64, kSub = kPosTile / kKv4Tile;
constexpr int kSoftWarps = 8, kProdWarps = 8, kProd = 16 * kProdWarps;  // kProd: threads of a group of four warps
constexpr int kChunkThreads = 32 * (kSoftWarps + kProdWarps + 4);  // five warpgroups
// Registers per thread: the block starts with kRegsStart and its warpgroups trade them (4 x 512 rows, STAGE_F32: 57.6 us with
// these, 57.4 with 152, 64, 48, 59.4 with 136, 80, 48; 2 x 1024 rows, STAGE_BF16: 342, 348, 350).
constexpr int kRegsStart = 96, kRegsSoft = 144, kRegsProd = 72, kRegsRest = 48;
static_assert(32 * (kSoftWarps * kRegsSoft + kProdWarps * kRegsProd + 4 * kRegsRest) <= kChunkThreads * kRegsStart, "the trade adds up");
static_assert(kChunkThreads * kRegsStart <= 65536 && kSoftWarps % 4 == 0 && kProdWarps % 4 == 0, "whole warpgroups");
constexpr int kChain = 128;  // tiles, a power of two
constexpr int kInfo = 16;  // ring of what the tiles' producers tell the softmax
// The largest probability (times its power of V) lies at 2^top when the reference is set, and may grow by 2^slack before
// it is set again: fp16 ends at 2^16.  With one fp16 value per probability fewer changes count more than the range below.
template <int NP>
constexpr float kChunkTop = NP == 2 ? 11.f : 7.f;
template <int NP>
constexpr float kChunkSlack = 15.f - kChunkTop<NP>;
constexpr uint64_t kWaitNs = 1000000000ull, kDrainNs = 200000000ull;
constexpr int kRaw = 4;    // packed tiles in shared memory
constexpr uint32_t kTmemCols = 512, kColQ = 0, kColS = 128, kColP = 256, kColO = 384;

struct ChunkBars {
  uint64_t q_full, raw_full[kRaw], raw_empty[kRaw], k_full[3], k_empty[3], v_full[3], v_empty[3],
      s_full[2], p_full[2], o_full[2], drain;
  uint64_t pair_q[2], pair_s[2][2], pair_p[2][2], pair_o[2][2];  // of the kernel with two row tiles: [tile][buffer]
};

// What a call has, the same for all its items: read from the kernel's parameters, so that it takes no registers.
struct ChunkArgs : Kv4AttnArgs {
  long long count;       // numbers of items, at most kKv4ChunkItems; those of sequences without such rows are none
  int group, row_tiles;  // query heads per KV head; row tiles of a sequence at the call's bounds
  int parts;             // of a row tile's positions
  int stall;             // copy no tile: the waits run out
};

struct ChunkItem {
  long long number;
  int seq, head, row0;             // sequence, KV head, first row
  int start, tokens, len, ncols;   // first query token of the sequence, its tokens, its positions, its rows
  int lim_hi, t0, nt;              // positions that some row sees; the first of the item's tiles and how many they are
};

// Items of ROWS rows: row tiles from the last (which sees most) down, then KV heads, then sequences, then the parts of
// their positions, dealt to the CTAs forth and back: c, 2 G - 1 - c, 2 G + c, ... of G, so that nobody has the longest of
// every round (4 x 512 rows, STAGE_F32: 64 us, 66 dealt forth alone).  Every warp goes through them for itself.
// kParts: there are parts.  kLoose: at the call's bounds most numbers are no items, because the bounds are loose or one sequence of
// many has most of the tokens; then a warp looks for its next item 32 numbers at a time (1 sequence of 2000 tokens among 4096 of
// one, STAGE_F32: 1.7 ms, 6.0 one by one; 1 of 512 among 64: 49 us, 62).  As kernels of their own: what a loop over tiles has to keep
// counts, the kernels live off their last registers (2 x 1024 rows of STAGE_BF16: 346 us, 391 with this search, which they do not need).
enum { kTight, kParts, kLoose };
template <int ROWS, int MODE>
struct ChunkItems {
  static constexpr bool SPLIT = MODE == kParts;
  const ChunkArgs& a;
  ChunkItem it;
  int round = 0;
  __device__ __forceinline__ explicit ChunkItems(const ChunkArgs& args) : a(args) {}
  // Takes number w apart; false if its sequence has no such rows.
  __device__ __forceinline__ bool at(long long w) {
    const int parts = SPLIT ? a.parts : 1;
    const uint32_t per = (uint32_t)a.c.n_kv_heads * a.n_seqs * parts, back = (uint32_t)w / per;  // kKv4ChunkItems bounds them
    const int row_tile = a.row_tiles - 1 - (int)back, rest = (int)((uint32_t)w - back * per), part = rest % parts, row = rest / parts;
    const int seq = row / a.c.n_kv_heads, row0 = row_tile * ROWS;
    int start;
    const int tokens = seq_tokens(a, seq, &start), ncols = min(tokens, a.max_q) * a.group;
    if (row0 >= ncols) return false;
    it.number = w;
    it.seq = seq;
    it.head = row - seq * a.c.n_kv_heads;
    it.row0 = row0;
    it.start = start;
    it.tokens = tokens;
    it.len = seq_positions(a, seq);
    it.ncols = ncols;
    it.lim_hi = seen(min(ncols, row0 + ROWS) - 1);
    const long long nt = (it.lim_hi + kPosTile - 1) / kPosTile;
    it.t0 = (int)(nt * part / parts);
    it.nt = (int)(nt * (part + 1) / parts) - it.t0;
    return true;
  }
  __device__ __forceinline__ long long dealt(int r) const {
    return (long long)r * gridDim.x + (r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  }
  // The CTA's next item; false behind the last.  kLoose: the whole warp.
  __device__ __forceinline__ bool next() {
    while (true) {
      const long long w = dealt(round);
      if (w >= a.count) return false;
      ++round;
      if (at(w)) return true;
      if constexpr (MODE == kLoose)
        for (uint32_t found = 0; !found && dealt(round) < a.count;) {
          const long long mine = dealt(round + (int)(threadIdx.x & 31));
          found = __ballot_sync(0xffffffffu, mine < a.count && live((uint32_t)mine));
          round += found ? __ffs(found) - 1 : 32;
        }
    }
  }
  // Whether number w is an item (of a sequence that has such rows).
  __device__ __forceinline__ bool live(uint32_t w) const {
    const uint32_t per = (uint32_t)a.c.n_kv_heads * a.n_seqs, back = w / per;
    int start;
    const int tokens = seq_tokens(a, (int)((w - back * per) / (uint32_t)a.c.n_kv_heads), &start);
    return (a.row_tiles - 1 - (int)back) * ROWS < min(tokens, a.max_q) * a.group;
  }
  // Positions that the item's sequence shows to row r.
  __device__ __forceinline__ int seen(int r) const { return max(0, it.len - it.tokens + r / a.group + 1); }
};

// Prepared scales of a tile: [position][block] fp16, each eight positions a padding further, for the banks.
__host__ __device__ constexpr int scale_place(int D, int pos) { return pos * (D / 16) + (pos >> 3) * (D / 8); }
constexpr int kWide = 16, kSpread = 32;
constexpr int kScaleBytes = scale_place(128, kPosTile);

struct alignas(16) ChunkMisc {
  ChunkBars bar;
  float v_exp[kInfo], v_inv[kInfo];  // E_v; 2^-E_v (0 and 0 where each position has its own)
  alignas(16) float k_pos_pow[kInfo][kPosTile];
  alignas(16) float v_pos_exp[kInfo][kPosTile];  // read in 16-byte pieces
  alignas(16) float v_pos_inv[kInfo][kPosTile];  // E_v and 2^-E_v of each position
  alignas(16) unsigned char k_scale[kProdWarps][kScaleBytes], v_scale[kProdWarps][kScaleBytes];  // a tile's scales as the products
                                                                                                 // take them, one copy per warp
  int absent[kInfo];                               // bit i: the tile's i-th 16 positions are not there
  int odd[kInfo];                                  // the same, and kWide, kSpread: its positions have powers of K, of V of their own
  int bad[kInfo];                                  // whether some V scale is no number
  int first_bad[kInfo][4];                         // per block of dims: the first such position
  float top[2][2][kRowsTile], q_top[2][kRowsTile]; // [tile parity][half][row]
  uint32_t tmem;
  int abort;
};

static_assert(offsetof(ChunkMisc, v_pos_exp) % 16 == 0 && offsetof(ChunkMisc, v_pos_inv) % 16 == 0, "vector reads");

// Shared memory: KS stages of K and of V operands behind QB bytes of q, or of the warps' places to turn rows (kTurn each).
constexpr int kTurn = 32 * 128;
template <int D, int NKV, int KS, int QB>
struct ChunkLayout {
  static constexpr int k_part = kPosTile * D * 2, v_part = D * kPosTile * 2;
  static constexpr int sub_stride = kv4_tile_bytes(D) + 32, stage_bytes = kSub * sub_stride;
  static constexpr int off_k = QB, off_v = off_k + KS * NKV * k_part, off_raw = off_v + KS * NKV * v_part;
  static constexpr int off_misc = off_raw + kRaw * stage_bytes;
  static_assert(off_k % 1024 == 0 && off_v % 1024 == 0 && k_part % 1024 == 0 && v_part % 1024 == 0, "swizzled tiles");
  static_assert(off_raw % 16 == 0 && stage_bytes % 16 == 0 && sub_stride % 16 == 0 && off_misc % 16 == 0, "16-byte pieces");
  static constexpr int bytes = off_misc + (int)sizeof(ChunkMisc) + 1024;  // and the alignment to 1024
};

// Bounded wait that also gives up as soon as another role of the CTA has given up.
__device__ __forceinline__ bool cwait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_ns() - t0 > kWaitNs) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// A softmax thread works on a row, but 32 rows in one access are 32 lines: rows go between global memory and their
// threads through kTurn bytes of the warp's shared memory, CH 16-byte pieces of a row at a time, swizzled, and a line is
// touched once (4 x 512 rows, STAGE_F32: 66 us, 71 with a row per lane).  `off`: where the lane's row begins behind `base`, in
// bytes; below 0: it is none.  The kernel for STAGE_BF16, whose items are longer, does without: there it cost registers, and
// 397 us became 355 without it (2 x 1024 rows).
template <int CH>
__device__ __forceinline__ unsigned char* turn_place(unsigned char* turn, int row, int piece) {
  return turn + (row * CH + (piece ^ (CH == 8 ? row & 7 : (row >> 1) & 3))) * 16;
}
template <int CH, int PASSES>
__device__ __forceinline__ void rows_in(unsigned char* turn, const void* base, long long off, uint4 (&own)[PASSES * CH]) {
  const int lane = threadIdx.x & 31;
  uint4 v[PASSES][CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const long long at = __shfl_sync(0xffffffffu, off, i * (32 / CH) + lane / CH);
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
      v[p][i] = at >= 0 ? *reinterpret_cast<const uint4*>((const char*)base + at + p * (16 * CH) + lane % CH * 16) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
#pragma unroll
    for (int i = 0; i < CH; ++i) *reinterpret_cast<uint4*>(turn_place<CH>(turn, i * (32 / CH) + lane / CH, lane % CH)) = v[p][i];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < CH; ++j) own[p * CH + j] = *reinterpret_cast<const uint4*>(turn_place<CH>(turn, lane, j));
    __syncwarp();
  }
}
template <int CH>
__device__ __forceinline__ void rows_out(unsigned char* turn, void* base, long long off, const uint4* own) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < CH; ++j) *reinterpret_cast<uint4*>(turn_place<CH>(turn, lane, j)) = own[j];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int row = i * (32 / CH) + lane / CH;
    const long long at = __shfl_sync(0xffffffffu, off, row);
    const uint4 v = *reinterpret_cast<const uint4*>(turn_place<CH>(turn, row, lane % CH));
    if (at >= 0) *reinterpret_cast<uint4*>((char*)base + at + lane % CH * 16) = v;
  }
  __syncwarp();
}

// Partial results, where a row tile's positions are shared out: per item and row the sums (float32, not divided), and
// the reference and the sum that divides them.  Before these, and without parts, the chains' sums lie there.
__device__ __forceinline__ float* part_row(void* ws, long long number, int rows, int row, int D) {
  return reinterpret_cast<float*>((char*)ws + kKv4CounterBytes) + (number * rows + row) * D;
}
__device__ __forceinline__ float2* part_ml(void* ws, long long count, long long number, int rows, int row, int D) {
  return reinterpret_cast<float2*>(part_row(ws, count, rows, 0, D)) + number * rows + row;
}

// END: the sums of a row's dims from `place` (TMEM) on are added to those of the chains that are done (`first`: there are none
// yet), and set to 0; else those are added to them.  They lie at the partial results' place `number` of `count`, the reference
// that they are of beside them, one for each half of the row's dims.  The whole warp.  A function of its own: inside the
// kernels, which live off their last registers, it made 2 x 1024 rows of STAGE_BF16 take 398 us instead of 349.
template <int D, int ROWS, int DIMS, bool END>
__device__ __noinline__ void chain_sums(void* ws, long long number, long long count, int row, int half, uint32_t place, float ref, bool first) {
  float* done = part_row(ws, number, ROWS, row, D) + half * DIMS;
  float* done_ref = &part_ml(ws, count, number, ROWS, row, D)->x + half;
  const float old = first ? 0.f : *done_ref, factor = first ? 0.f : old == ref ? 1.f : exp2_approx(old - ref);
#pragma unroll 1
  for (int d = 0; d < DIMS; d += 16) {
    uint32_t r[16];
    tmem_ld16(place + d, r);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      float4* at = reinterpret_cast<float4*>(done + d + j);
      float4 v = factor != 0.f ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
      v = make_float4(fmaf(v.x, factor, __uint_as_float(r[j])), fmaf(v.y, factor, __uint_as_float(r[j + 1])),
                      fmaf(v.z, factor, __uint_as_float(r[j + 2])), fmaf(v.w, factor, __uint_as_float(r[j + 3])));
      if (END) *at = v;
      r[j] = END ? 0 : __float_as_uint(v.x), r[j + 1] = END ? 0 : __float_as_uint(v.y);
      r[j + 2] = END ? 0 : __float_as_uint(v.z), r[j + 3] = END ? 0 : __float_as_uint(v.w);
    }
    tmem_st16(place + d, r);
  }
  tmem_wait_st();
  if (END) *done_ref = ref;
}

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// The codes of (1024 + c) and (1024 + 16 c) pairs minus 8.
__device__ __forceinline__ __half2 code_low(uint32_t x, uint32_t ex) {
  return __hadd2(as_h2(and_or(x, 0x000f000fu, ex)), __floats2half2_rn(-1032.f, -1032.f));
}
__device__ __forceinline__ __half2 code_high(uint32_t x, uint32_t ex) {
  return __hfma2(as_h2(and_or(x, 0x00f000f0u, ex)), __floats2half2_rn(0.0625f, 0.0625f), __floats2half2_rn(-72.f, -72.f));
}

// 2^k in both halves, k in [-14, 15].
__device__ __forceinline__ __half2 half_power(int k) { return __half2half2(__ushort_as_half((uint16_t)((15 + k) << 10))); }

// K's scales from 4096 on (fp16 bits from here on) are divided by a power of two: e of a position with the largest scale `top`.
constexpr uint32_t kBigScale = 27u << 10;
__device__ __forceinline__ int k_power(uint32_t top) { return max(0, (int)min(top >> 10, 30u) - 26); }
// V's are multiplied by 2^k twice (once would not reach: 2^26 for subnormal ones): k of the largest scale `top`, for 2^10 .. 2^12.
__device__ __forceinline__ int v_power(uint32_t top) { return (26 - (int)(top >> 10)) >> 1; }
__device__ __forceinline__ uint32_t larger_half(__half2 m) { return max(as_u32(m) >> 16, as_u32(m) & 0xffffu); }

// ---------------- what both kernels have ----------------

__device__ void chunk_init(ChunkMisc& M) {
  ChunkBars& B = M.bar;
  for (int i = 0; i < kRaw; ++i) {
    mbar_init(&B.raw_full[i], 1);
    mbar_init(&B.raw_empty[i], kProd);
  }
  for (int i = 0; i < 3; ++i) {
    mbar_init(&B.k_full[i], kProd);
    mbar_init(&B.v_full[i], kProd);
    mbar_init(&B.k_empty[i], 1);
    mbar_init(&B.v_empty[i], 1);
  }
  mbar_init(&B.q_full, 32 * kSoftWarps);
  for (int i = 0; i < 2; ++i) {
    mbar_init(&B.s_full[i], 2);
    mbar_init(&B.o_full[i], 2);
    mbar_init(&B.p_full[i], 32 * kSoftWarps);
    mbar_init(&B.pair_q[i], 16 * kSoftWarps);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&B.pair_s[i][b], 2);
      mbar_init(&B.pair_o[i][b], 2);
      mbar_init(&B.pair_p[i][b], 16 * kSoftWarps);
    }
  }
  mbar_init(&B.drain, 1);
  M.abort = 0;
  for (int i = 0; i < kInfo; ++i) {
    M.bad[i] = 0;
    for (int b = 0; b < 4; ++b) M.first_bad[i][b] = INT_MAX;
  }
  mbar_fence_init();
}

// Expansion, by two groups of four warps: group g has the tiles n with n % 2 = g, in KS stages of operands.
template <int D, int NKV, int NP, int KS, typename L, int ROWS, int MODE>
__device__ __forceinline__ void chunk_expand(unsigned char* sm, ChunkMisc& M, ChunkItems<ROWS, MODE>& items) {
  constexpr int NB = D / 32, HALF = kv4_half(D), CODES = kv4_codes(D);
  ChunkBars& B = M.bar;
  volatile int* abort_flag = &M.abort;
  const ChunkItem& it = items.it;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group_of = (warp - kSoftWarps) >> 2, p = tid - 32 * (kSoftWarps + 4 * group_of), pw = p >> 5;
  const uint32_t ex = exponent_bits();
  bool ok = true;  // a warp in which a wait has run out leaves as a whole
  int n = 0;
  for (; ok && items.next(); n += it.nt)
  for (int i = (n & 1) == group_of ? 0 : 1; i < it.nt; i += 2) {
    const int ni = n + i, st = ni % KS, rs = ni & (kRaw - 1), inf = ni & (kInfo - 1), lim_hi = it.lim_hi;
    ok = __all_sync(0xffffffffu, cwait(&B.raw_full[rs], (uint32_t)(ni / kRaw) & 1u, abort_flag));
    if (!ok) break;
    const int absent = M.absent[inf];
    const unsigned char* raw = sm + L::off_raw + rs * L::stage_bytes;
    const int pos0 = (it.t0 + i) * kPosTile;

    // the scales, every warp for itself: a lane has two neighbouring positions.  Those that do not count read as 0
    int k_tile = 0;
    bool v_bad = false, k_big, v_spread = false;
    unsigned char *k_scale = M.k_scale[warp - kSoftWarps], *v_scale = M.v_scale[warp - kSoftWarps];
    {
      const int s = lane >> 3, at = pos0 + s * kKv4Tile + 2 * (lane & 7);
      const bool ok0 = !(absent >> s & 1) && at < lim_hi, ok1 = !(absent >> s & 1) && at + 1 < lim_hi;
      const unsigned char* base = raw + s * L::sub_stride + (lane & 7) * (4 * NB);
      uint32_t w[NB];  // words 0 .. NB / 2 - 1: the first position's
      auto load = [&](const unsigned char* from) {
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(from);
          w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(from);
          w[0] = u.x, w[1] = u.y;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (!(b < NB / 2 ? ok0 : ok1)) w[b] = 0;
      };
      auto largest = [&](int i) {  // of the first or the second position; NaN loses
        __half2 m = as_h2(w[i * (NB / 2)] & 0x7fff7fffu);
        if (NB == 4) m = __hmax2(m, as_h2(w[i * (NB / 2) + NB / 2 - 1] & 0x7fff7fffu));
        m = __hmax2(m, __floats2half2_rn(0.f, 0.f));
        return larger_half(m);
      };
      auto put = [&](unsigned char* to) {
        if constexpr (D == 128) *reinterpret_cast<uint4*>(to + scale_place(D, 2 * lane)) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(to + scale_place(D, 2 * lane)) = make_uint2(w[0], w[1]);
      };
      __syncwarp();  // the last tile's are read
      load(base + HALF + CODES + 16 + ((lane & 4) << 2));
#pragma unroll
      for (int b = 0; b < NB; ++b) v_bad |= (w[b] & 0x7c00u) == 0x7c00u || (w[b] & 0x7c000000u) == 0x7c000000u;
      v_bad = __any_sync(0xffffffffu, v_bad);
      if (v_bad) {  // noted, and taken for 0
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t ones = h ? 0x7c000000u : 0x7c00u;
            if ((w[b] & ones) == ones) {
              if (pw == 0) atomicMin(&M.first_bad[inf][2 * b % NB + h], at + (b >= NB / 2));
              w[b] &= h ? 0xffffu : 0xffff0000u;
            }
          }
      }
      const uint32_t top0 = largest(0), top1 = largest(1);
      int k0 = v_power(top0), k1 = v_power(top1);
      if (NP == 1) {
        const uint32_t high = __reduce_max_sync(0xffffffffu, max(top0, top1));
        const uint32_t low = __reduce_min_sync(0xffffffffu, min(top0 ? top0 : 0x7c00u, top1 ? top1 : 0x7c00u));  // 0 is of any size
        v_spread = (low >> 10) + 3 < high >> 10;
        k_tile = v_power(high);
        if (!v_spread) k0 = k1 = k_tile;
      }
      if ((NP == 2 || v_spread) && pw == 0) {
        *reinterpret_cast<float2*>(&M.v_pos_exp[inf][2 * lane]) = make_float2((float)(-2 * k0), (float)(-2 * k1));
        *reinterpret_cast<float2*>(&M.v_pos_inv[inf][2 * lane]) =
            make_float2(__uint_as_float((uint32_t)(127 + 2 * k0) << 23), __uint_as_float((uint32_t)(127 + 2 * k1) << 23));
      }
      const __half2 up0 = half_power(k0), up1 = half_power(k1);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const __half2 up = b < NB / 2 ? up0 : up1;
        w[b] = as_u32(__hmul2(__hmul2(as_h2(w[b]), up), up));
      }
      put(v_scale);

      load(base + CODES);
      k_big = __reduce_max_sync(0xffffffffu, max(largest(0), largest(1))) >= kBigScale;
      if (k_big) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int e = k_power(largest(i));
          if (pw == 0) M.k_pos_pow[inf][2 * lane + i] = __uint_as_float((uint32_t)(127 + e) << 23);
          const __half2 norm = half_power(-e);
#pragma unroll
          for (int b = i * (NB / 2); b < (i + 1) * (NB / 2); ++b)  // an infinity becomes NaN: a score of -infinity would drop its position
            w[b] = as_u32(__hmul2(__hfma2(as_h2(w[b]), __floats2half2_rn(0.f, 0.f), as_h2(w[b])), norm));
        }
      }
      put(k_scale);
    }
    __syncwarp();  // the prepared scales
    // K: 64 positions x 4 x (the word of eight dims of every block)
    if (ni >= KS) ok = __all_sync(0xffffffffu, cwait(&B.k_empty[st], (uint32_t)(ni / KS + 1) & 1u, abort_flag));
    if (!ok) break;
    if (p == 0) {
      M.odd[inf] = absent | (k_big ? kWide : 0) | (v_spread ? kSpread : 0);
      if (NP == 1) {
        M.v_exp[inf] = v_spread ? 0.f : (float)(-2 * k_tile);
        M.v_inv[inf] = v_spread ? 0.f : __uint_as_float((uint32_t)(127 + 2 * k_tile) << 23);
      }
      M.bad[inf] = v_bad;
      // For tile n + kRaw, which no warp has begun: its copy waits until every warp of the group has read tile n.  The
      // entry's last tile, n + kRaw - kInfo, was read by the softmax before it handed on the probabilities of a tile whose
      // products the scores of tile n - KS waited for; and those are done.
      const int next = (inf + kRaw) & (kInfo - 1);
      for (int b = 0; b < 4; ++b) M.first_bad[next][b] = INT_MAX;
    }
    unsigned char* kt = sm + L::off_k + st * NKV * L::k_part;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tig = lane & 3, pos = ((lane >> 2) & 1) * 4 + ((lane >> 3) & 3) + 8 * (pw + 4 * j), s = pos >> 4;
      const unsigned char* src = raw + s * L::sub_stride;
      uint32_t w[NB], sc[NB / 2];
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(src + (pos & 15) * (D / 2) + tig * 16);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        const uint2 v = *reinterpret_cast<const uint2*>(k_scale + scale_place(D, pos));
        sc[0] = v.x, sc[1] = v.y;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(src + (pos & 15) * (D / 2) + tig * 8);
        w[0] = u.x, w[1] = u.y;
        sc[0] = *reinterpret_cast<const uint32_t*>(k_scale + scale_place(D, pos));
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const __half2 s2 = as_h2(__byte_perm(sc[b / 2], 0, b & 1 ? 0x3232 : 0x1010));
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t x = t < 2 ? w[b] : w[b] >> 8;
          const __half2 n = t & 1 ? code_high(x, ex) : code_low(x, ex);
          const __half2 h = __hmul2(n, s2);
          hi[t] = as_u32(h);
          if (NKV == 2) lo[t] = as_u32(__hfma2(n, s2, __hneg2(h)));
        }
        unsigned char* at = kt + (b >> 1) * (kPosTile * 128) + sw128_offset(pos, 32 * (b & 1) + 8 * tig);
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (NKV == 2) *reinterpret_cast<uint4*>(at + L::k_part) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    fence_async_smem();
    mbar_arrive(&B.k_full[st]);

    // V: a thread has eight positions (chunk) and two of the four dims 4 gid .. + 3 of every block.  Eight lanes with the
    // same dims and different chunks read 16 bytes each from places 16 bytes apart modulo 128 (hence the paddings
    // of the raw tiles) and write a whole row of 64 positions
    if (ni >= KS) ok = __all_sync(0xffffffffu, cwait(&B.v_empty[st], (uint32_t)(ni / KS + 1) & 1u, abort_flag));
    if (!ok) break;
    {
      unsigned char* vt = sm + L::off_v + st * NKV * L::v_part;
      constexpr int VB = NKV == 1 ? NB : NB / 2;  // blocks at a time, for the registers
      const int chunk = lane & 7, dsel = (lane >> 3) & 1, gid = pw * 2 + (lane >> 4), s = chunk >> 1, h = chunk & 1;
      const unsigned char* src = raw + s * L::sub_stride + HALF;
      const unsigned char* codes = src + h * (CODES / 2 + 16) + gid * (D / 2);
      const unsigned char* scales = v_scale + scale_place(D, 8 * chunk);
#pragma unroll 1
      for (int b0 = 0; b0 < NB; b0 += VB) {
      uint32_t hi[VB][2][4], lo[VB][2][4];
#pragma unroll
      for (int tig = 0; tig < 4; ++tig) {
        constexpr int W = (VB + 1) / 2;  // words of a position's blocks
        uint32_t w[2][W], sc[2][W];      // of the first and the second position
        if constexpr (D == 128 && VB == 4) {
          const uint4 u = *reinterpret_cast<const uint4*>(codes + tig * 16);
          w[0][0] = u.x, w[0][1] = u.y, w[1][0] = u.z, w[1][1] = u.w;
          const uint4 v = *reinterpret_cast<const uint4*>(scales + tig * 16);
          sc[0][0] = v.x, sc[0][1] = v.y, sc[1][0] = v.z, sc[1][1] = v.w;
        } else if constexpr (D == 128) {
          w[0][0] = *reinterpret_cast<const uint32_t*>(codes + tig * 16 + b0 * 2);
          w[1][0] = *reinterpret_cast<const uint32_t*>(codes + tig * 16 + 8 + b0 * 2);
          sc[0][0] = *reinterpret_cast<const uint32_t*>(scales + tig * 16 + b0 * 2);
          sc[1][0] = *reinterpret_cast<const uint32_t*>(scales + tig * 16 + 8 + b0 * 2);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(codes + tig * 8);
          w[0][0] = u.x >> (16 * b0), w[1][0] = u.y >> (16 * b0);
          const uint2 v = *reinterpret_cast<const uint2*>(scales + tig * 8);
          sc[0][0] = v.x >> (16 * b0), sc[1][0] = v.y >> (16 * b0);
        }
#pragma unroll
        for (int b = 0; b < VB; ++b) {
          const __half2 s2 = as_h2(__byte_perm(sc[0][b / 2], sc[1][b / 2], b & 1 ? 0x7632 : 0x5410));
          // byte dsel of the block's two bytes, of both positions
          const uint32_t x = __byte_perm(w[0][b / 2], w[1][b / 2], (b & 1 ? 0x6622 : 0x4400) + dsel * 0x1111);
          const __half2 n0 = code_low(x, ex), n1 = code_high(x, ex);
          const __half2 h0 = __hmul2(n0, s2), h1 = __hmul2(n1, s2);
          hi[b][0][tig] = as_u32(h0);
          hi[b][1][tig] = as_u32(h1);
          if (NKV == 2) {
            lo[b][0][tig] = as_u32(__hfma2(n0, s2, __hneg2(h0)));
            lo[b][1][tig] = as_u32(__hfma2(n1, s2, __hneg2(h1)));
          }
        }
      }
      if (b0 + VB == NB) mbar_arrive(&B.raw_empty[rs]);
#pragma unroll
      for (int b = 0; b < VB; ++b)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int dim = 32 * (b0 + b) + 4 * gid + 2 * dsel + k;
          unsigned char* at = vt + sw128_offset(dim, 8 * chunk);
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[b][k][0], hi[b][k][1], hi[b][k][2], hi[b][k][3]);
          if (NKV == 2) *reinterpret_cast<uint4*>(at + L::v_part) = make_uint4(lo[b][k][0], lo[b][k][1], lo[b][k][2], lo[b][k][3]);
        }
      }
    }
    fence_async_smem();
    mbar_arrive(&B.v_full[st]);
  }
}

// Copies of the packed tiles, by one thread (kLoose: of a whole warp, which looks for the items).
template <int D, typename L, int ROWS, int MODE>
__device__ __forceinline__ void chunk_copy(unsigned char* sm, ChunkMisc& M, ChunkItems<ROWS, MODE>& items) {
  constexpr int TILE = kv4_tile_bytes(D), HALF = kv4_half(D), CODES = kv4_codes(D);
  ChunkBars& B = M.bar;
  volatile int* abort_flag = &M.abort;
  const ChunkArgs& a = items.a;
  const ChunkItem& it = items.it;
  const int tpp = a.c.page_len / kKv4Tile;
  bool ok = true;
  int n = 0;
  for (; (MODE == kLoose ? __all_sync(0xffffffffu, ok) : ok) && items.next();) {
    if (MODE == kLoose && (threadIdx.x & 31)) continue;
    const int n16 = (it.lim_hi + kKv4Tile - 1) / kKv4Tile;
    const int* trow = a.table + (long long)it.seq * a.table_stride;
    // the pages of a tile are asked for a tile ahead; places go on without a division
    int ids[kSub], places[kSub], next_t = it.t0 * kSub, next_page = next_t / tpp, next_place = next_t - next_page * tpp;
    auto ask = [&]() {
#pragma unroll
      for (int s = 0; s < kSub; ++s) {
        ids[s] = next_t < n16 ? trow[next_page] : -1;
        places[s] = next_place;
        ++next_t;
        if (++next_place == tpp) {
          next_place = 0;
          ++next_page;
        }
      }
    };
    ask();
    for (int i = 0; i < it.nt; ++i, ++n) {
      const int rs = n & (kRaw - 1);
      ok = n < kRaw || cwait(&B.raw_empty[rs], (uint32_t)(n / kRaw + 1) & 1u, abort_flag);
      if (!ok) break;
      unsigned char* raw = sm + L::off_raw + rs * L::stage_bytes;
      int absent = 0, here = 0;
#pragma unroll
      for (int s = 0; s < kSub; ++s) {
        const bool there = ids[s] >= 0 && ids[s] < a.c.n_pages;
        absent |= there ? 0 : 1 << s;
        here += there;
      }
      M.absent[n & (kInfo - 1)] = absent;
      mbar_arrive_expect_tx(&B.raw_full[rs], here * TILE);
      // V's second half, and the second half of its scales, go 16 bytes on each: see their reads
      constexpr int cut = HALF + CODES / 2, cut2 = HALF + CODES + kv4_scales(D) / 2;
#pragma unroll
      for (int s = 0; s < kSub; ++s)
        if (!(absent >> s & 1)) {
          const uint8_t* src = a.c.data + (((long long)ids[s] * a.c.n_kv_heads + it.head) * tpp + places[s]) * TILE;
          unsigned char* dst = raw + s * L::sub_stride;
          bulk_g2s(dst, src, cut, &B.raw_full[rs]);
          bulk_g2s(dst + cut + 16, src + cut, cut2 - cut, &B.raw_full[rs]);
          bulk_g2s(dst + cut2 + 32, src + cut2, TILE - cut2, &B.raw_full[rs]);
        }
      ask();
    }
  }
  // Nothing may still be landing in shared memory when the CTA leaves, whoever has given up, be it after this (n: the copying thread's)
  for (int i = max(0, n - kRaw); i < n; ++i) mbar_wait(&B.raw_full[i & (kRaw - 1)], (uint32_t)(i / kRaw) & 1u, kDrainNs);
}

template <int D, int NQ, int NKV, int NP, int MODE>
__global__ void __launch_bounds__(kChunkThreads, 1) kv4_chunk_kernel(const ChunkArgs a) {
  constexpr bool SPLIT = MODE == kParts;
  using L = ChunkLayout<D, NKV, 2, kSoftWarps * kTurn>;
  constexpr int HD = D / 2;  // dims of a softmax thread
  constexpr bool F32 = NP == 2;
  extern __shared__ unsigned char chunk_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)chunk_raw + 1023) & ~(uintptr_t)1023);
  ChunkMisc& M = *reinterpret_cast<ChunkMisc*>(sm + L::off_misc);
  ChunkBars& B = M.bar;
  volatile int* abort_flag = &M.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  ChunkItems<kRowsTile, MODE> items(a);
  const ChunkItem& it = items.it;

  if (tid == 0) chunk_init(M);
  if (warp == 0) {
    tmem_alloc(&M.tmem, kTmemCols);
    tmem_relinquish();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = M.tmem;

  if (warp >= kSoftWarps && warp < kSoftWarps + kProdWarps) {
    // ---------------- producers ----------------
    regs_down<kRegsProd>();
    chunk_expand<D, NKV, NP, 2, L>(sm, M, items);
  } else if (warp >= kSoftWarps + kProdWarps) {
    regs_down<kRegsRest>();
    if (warp == kSoftWarps + kProdWarps + 1 && (MODE == kLoose || lane == 0)) {
      // ---------------- copies ----------------
      if (!a.stall) chunk_copy<D, L>(sm, M, items);
    }
    if (warp == kSoftWarps + kProdWarps) {
      // ---------------- products ----------------
      // The whole warp goes through the loops and one elected thread issues: addresses and descriptors then are uniform
      // values, which the instructions take as they are.
      const bool leader = elect_one();
      constexpr uint32_t id_s = idesc_f16_f32(kRowsTile, kPosTile), id_o = idesc_f16_f32(kRowsTile, D);
      const uint64_t kd = desc_sw128(smem_u32(sm + L::off_k)), vd = desc_sw128(smem_u32(sm + L::off_v));
      uint32_t s_st = 0, s_ph = 0, o_st = 0, o_ph = 0;  // stage and parity of the next tile's scores and outputs
      auto scores = [&]() {
        if (!__all_sync(0xffffffffu, cwait(&B.k_full[s_st], s_ph, abort_flag))) return false;
        tc_fence_after();
        const uint64_t kb = kd + s_st * (uint32_t)(NKV * L::k_part >> 4);
        const uint32_t d = tmem + kColS + s_st * kPosTile;
        if (leader) {
#pragma unroll
          for (int part = NQ + NKV - 2; part >= 0; --part)  // [high low,] [low high,] high high
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              umma_f16_ts(d, tmem + kColQ + (NQ == 2 && part == 1 ? D / 2 : 0) + ks * 8,
                          kb + (((part > 0 && part == NQ ? L::k_part : 0) + (ks >> 2) * (kPosTile * 128) + (ks & 3) * 32) >> 4),
                          id_s, part < NQ + NKV - 2 || ks ? 1u : 0u);
          umma_commit(&B.k_empty[s_st]);
          umma_commit(&B.s_full[s_st]);
          mbar_arrive(&B.s_full[s_st]);  // hands on what the producers wrote beside the tile
        }
        __syncwarp();
        s_st ^= 1;
        s_ph ^= s_st ? 0u : 1u;
        return true;
      };
      bool ok = true;
      uint32_t q_ph = 0;
      for (; ok && items.next();) {
        if (it.nt == 0) continue;  // its q is not waited for, and not announced
        ok = __all_sync(0xffffffffu, cwait(&B.q_full, q_ph, abort_flag));
        q_ph ^= 1;
        if (!ok) break;
        tc_fence_after();
        ok = scores();
        if (ok && it.nt > 1) ok = scores();
        for (int i = 0; ok && i < it.nt; ++i) {
          ok = __all_sync(0xffffffffu, cwait(&B.v_full[o_st], o_ph, abort_flag) && cwait(&B.p_full[o_st], o_ph, abort_flag));
          if (!ok) break;
          tc_fence_after();
          const uint64_t vb = vd + o_st * (uint32_t)(NKV * L::v_part >> 4);
          const uint32_t pc = tmem + kColP + o_st * 64;
          const uint32_t again = NP == 1 && i > 0 ? 1u : 0u;
          if (leader) {
#pragma unroll
            for (int part = NP + NKV - 2; part >= 0; --part)
#pragma unroll
              for (int ks = 0; ks < kPosTile / 16; ++ks)
                umma_f16_ts(tmem + kColO, pc + (NP == 2 && part == 1 ? 32 : 0) + ks * 8,
                            vb + (((part > 0 && part == NP ? L::v_part : 0) + ks * 32) >> 4), id_o,
                            part < NP + NKV - 2 || ks ? 1u : again);
            umma_commit(&B.v_empty[o_st]);
            umma_commit(&B.o_full[o_st]);
            mbar_arrive(&B.o_full[o_st]);
          }
          __syncwarp();
          o_st ^= 1;
          o_ph ^= o_st ? 0u : 1u;
          // the softmax of tile i has read its scores: their place is free
          if (i + 2 < it.nt) ok = scores();
        }
      }
      if (leader) {  // the products finish before TMEM is released, whoever has given up waiting for them
        umma_commit(&B.drain);
        mbar_wait(&B.drain, 0u, kDrainNs);
      }
    }
  } else {
    // ---------------- softmax ----------------
    regs_up<kRegsSoft>();
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int row = 32 * (warp & 3) + lane, half = (warp >> 2) & 1;
    unsigned char* turn = sm + warp * kTurn;
    bool ok = true;
    int n = 0;
    for (; items.next(); n += it.nt) {
    const int nt = it.nt, lim_lo = items.seen(it.row0);  // positions that every row sees
    const int col = it.row0 + row;
    const bool live = col < it.ncols;
    const int col_k = col / a.group;
    const int lim = live ? items.seen(col) : 0;
    const long long elem = (long long)(it.head * a.group + col - col_k * a.group) * D + half * HD;
    // ---- q into TMEM: scaled by a power of two per row, high and low part; within eight dims in the order of the unpacked
    // codes (0, 4, 1, 5, 2, 6, 3, 7).  The last item's scores are done with its q: this thread has waited for them
    float zscale;
    {
      float q[HD / 8][8], top = 0.f;
      constexpr int W = HD * (F32 ? 4 : 2) / 16;  // 16-byte pieces of the thread's dims
      uint4 own[W];
      rows_in<W < 8 ? W : 8, W < 8 ? 1 : W / 8>(turn, a.q, live ? ((long long)(it.start + col_k) * a.q_stride + elem) * (F32 ? 4 : 2) : -1, own);
#pragma unroll
      for (int g = 0; g < HD / 8; ++g) {
        if constexpr (F32) {
          const uint4 lo = own[2 * g], hi = own[2 * g + 1];
          const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) q[g][i] = __uint_as_float(u[i]);
        } else {
          const uint32_t u[4] = {own[g].x, own[g].y, own[g].z, own[g].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = h2_to_f2(u[i]);
            q[g][2 * i] = f.x, q[g][2 * i + 1] = f.y;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(q[g][i]));
      }
      M.q_top[half][row] = top;
      named_bar(1 + (warp & 3), 64);
      top = fmaxf(top, M.q_top[half ^ 1][row]);
      const int e = top <= FLT_MAX ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 0;
      zscale = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(e - 13 + 127) << 23);
      const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
#pragma unroll
      for (int c = 0; c < HD / 2; c += 16) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int g = (c + j) >> 2, t = j & 3;
          const float x0 = q[g][t] * up, x1 = q[g][t + 4] * up;
          const __half2 h = __floats2half2_rn(x0, x1);
          const float2 f = __half22float2(h);
          hi[j] = as_u32(h);
          lo[j] = as_u32(__floats2half2_rn(x0 - f.x, x1 - f.y));
        }
        tmem_st16(lanes + kColQ + half * (HD / 2) + c, hi);
        if (NQ == 2) tmem_st16(lanes + kColQ + D / 2 + half * (HD / 2) + c, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      if (nt > 0) mbar_arrive(&B.q_full);
    }

    constexpr int NO = NP == 2 ? HD / 2 : 1;
    float2 o[NO];  // STAGE_F32: the sums over the tiles that are done
#pragma unroll
    for (int j = 0; j < NO; ++j) o[j] = make_float2(0.f, 0.f);
    float ref = -INFINITY, sum = 0.f;
    int nan_blocks = 0;  // the thread's blocks of dims in which its row sees a V scale that is no number
    auto products_done = [&](int i) {
      if (!__all_sync(0xffffffffu, cwait(&B.o_full[i & 1], (uint32_t)(i >> 1) & 1u, abort_flag))) return false;
      tc_fence_after();
      return true;
    };
    auto note_bad = [&](int i) {
      if (M.bad[i & (kInfo - 1)]) {
#pragma unroll
        for (int b = 0; b < HD / 32; ++b)
          if (M.first_bad[i & (kInfo - 1)][half * (HD / 32) + b] < lim) nan_blocks |= 1 << b;
      }
    };
    // adds a tile's sums to the registers
    auto collect = [&]() {
      if constexpr (NP == 2) {
#pragma unroll
        for (int c = 0; c < HD; c += 32) {
          uint32_t r[32];
          tmem_ld32(lanes + kColO + half * HD + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[c / 2 + j] = add2(o[c / 2 + j], make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])));
        }
      }
    };
    for (int i = 0; i < nt;) {  // STAGE_F16: chains of tiles
    if (NP == 1 && i > 0) {
      ok = ok && products_done(n + i - 1);
      if (ok) chain_sums<D, kRowsTile, HD, true>(a.ws, SPLIT ? it.number : (long long)blockIdx.x, SPLIT ? a.count : (long long)gridDim.x, row, half, lanes + kColO + half * HD, ref, i == kChain);
    }
    for (const int end = NP == 1 ? min(nt, i + kChain) : nt; i < end; ++i) {
      const int ni = n + i, st = ni & 1, inf = ni & (kInfo - 1);
      // S of tile i is there, and so is the product of tile i - 2, issued before it: P's place is free.  When a wait has run
      // out every thread still goes through the barriers, and does nothing else
      ok = ok && __all_sync(0xffffffffu, cwait(&B.s_full[st], (uint32_t)(ni >> 1) & 1u, abort_flag));
      if (!ok) {
        named_bar(1 + (warp & 3), 64);
        continue;
      }
      tc_fence_after();
      uint32_t s[32];
      tmem_ld32(lanes + kColS + st * kPosTile + half * 32, s);
      float f = zscale;
      const float ev = NP == 2 ? 0.f : M.v_exp[inf], v_inv = NP == 2 ? 1.f : M.v_inv[inf];
      const int odd = M.odd[inf];
      if (i >= 2) note_bad(ni - 2);
      tmem_wait_ld();
      const int pos0 = (it.t0 + i) * kPosTile + 32 * half;
      if (pos0 + 32 > lim_lo || odd) {
        if (odd & kWide) {
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) * M.k_pos_pow[inf][32 * half + j]);
        }
        if (NP == 1 && (odd & kSpread)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(fmaf(__uint_as_float(s[j]), f, M.v_pos_exp[inf][32 * half + j]));
          f = 1.f;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (pos0 + j >= lim || (odd >> (2 * half + (j >> 4)) & 1)) s[j] = 0xff800000u;
      }
      // exponents in base 2; STAGE_F32: with each position's power of V
      float most = -INFINITY;
      if constexpr (NP == 2) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 e4 = *reinterpret_cast<const float4*>(&M.v_pos_exp[inf][32 * half + j]);
          const float2 w0 = fma2(make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), make_float2(f, f), make_float2(e4.x, e4.y));
          const float2 w1 = fma2(make_float2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), make_float2(f, f), make_float2(e4.z, e4.w));
          s[j] = __float_as_uint(w0.x), s[j + 1] = __float_as_uint(w0.y), s[j + 2] = __float_as_uint(w1.x), s[j + 3] = __float_as_uint(w1.y);
        }
      }
      {
        float m4[4];  // four chains
#pragma unroll
        for (int j = 0; j < 4; ++j) m4[j] = __uint_as_float(s[j]);
#pragma unroll
        for (int j = 4; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(s[j]));
        most = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        if (NP == 1) most = fmaf(most, f, ev);
      }
      M.top[st][half][row] = most;
      named_bar(1 + (warp & 3), 64);
      most = fmaxf(most, M.top[st][half ^ 1][row]);
      float keep = 1.f;
      if (most - kChunkTop<NP> > ref + kChunkSlack<NP>) {
        keep = exp2_approx(ref - (most - kChunkTop<NP>));
        ref = most - kChunkTop<NP>;
        sum *= keep;
      }
      const bool moved = __any_sync(0xffffffffu, keep != 1.f);
      if (NP == 2 && i > 0) {  // the last tile's sums leave TMEM before this one's products
        ok = products_done(ni - 1);
        if (ok) collect();
      }
      if (NP == 2 && moved) {
#pragma unroll
        for (int j = 0; j < NO; ++j) o[j] = mul2(o[j], make_float2(keep, keep));
      }
      if (NP == 1 && moved && i > 0) {
        ok = products_done(ni - 1);
        if (ok) {
          const uint32_t at = lanes + kColO + half * HD;
#pragma unroll
          for (int c = 0; c < HD; c += 16) {
            uint32_t r[16];
            tmem_ld16(at + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * keep);
            tmem_st16(at + c, r);
          }
        }
      }
      const float c = ev - (ref == -INFINITY ? 0.f : ref);
      if (NP == 1 && (odd & kSpread)) {  // the sum by each position's power; the one below counts for 0 (v_inv)
#pragma unroll
        for (int j = 0; j < 32; ++j) sum += exp2_approx(__uint_as_float(s[j]) - M.v_pos_exp[inf][32 * half + j] + c);
      }
      float2 part4[4];  // four chains
#pragma unroll
      for (int j = 0; j < 4; ++j) part4[j] = make_float2(0.f, 0.f);
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 sj = make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
        const float2 z = NP == 2 ? add2(sj, make_float2(c, c)) : fma2(sj, make_float2(f, f), make_float2(c, c));
        const float2 x = make_float2(exp2_approx(z.x), exp2_approx(z.y));
        float2& part = part4[j & 3];
        part = NP == 2 ? fma2(x, *reinterpret_cast<const float2*>(&M.v_pos_inv[inf][32 * half + 2 * j]), part) : add2(part, x);
        const __half2 h = __floats2half2_rn(x.x, x.y);
        hi[j] = as_u32(h);
        if (NP == 2) {
          const float2 b = __half22float2(h);
          const float2 rest = add2(x, make_float2(-b.x, -b.y));
          lo[j] = as_u32(__floats2half2_rn(rest.x, rest.y));
        }
      }
      const float2 part = add2(add2(part4[0], part4[1]), add2(part4[2], part4[3]));
      sum = fmaf(part.x + part.y, v_inv, sum);
      tmem_st16(lanes + kColP + st * 64 + half * 16, hi);
      if (NP == 2) tmem_st16(lanes + kColP + st * 64 + 32 + half * 16, lo);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&B.p_full[st]);
    }
    }
    if (ok && nt > 0) {
      ok = products_done(n + nt - 1);
      if (ok && NP == 2) collect();
      if (ok && NP == 1 && nt > kChain) chain_sums<D, kRowsTile, HD, false>(a.ws, SPLIT ? it.number : (long long)blockIdx.x, SPLIT ? a.count : (long long)gridDim.x, row, half, lanes + kColO + half * HD, ref, false);
      if (nt > 1) note_bad(n + nt - 2);
      note_bad(n + nt - 1);
    }
    M.top[(n + nt) & 1][half][row] = sum;
    named_bar(1 + (warp & 3), 64);
    sum += M.top[(n + nt) & 1][half ^ 1][row];
    named_bar(1 + (warp & 3), 64);  // read before the next item writes there
    const float inv = !ok ? NAN : SPLIT ? 1.f : sum != 0.f ? 1.f / sum : 0.f;  // rows that could not be finished are NaN
    if (SPLIT && half == 0) *part_ml(a.ws, a.count, it.number, kRowsTile, row, D) = make_float2(ref, sum);
    // where the results go: the output, or (float32) the part's place
    void* out = SPLIT ? (void*)part_row(a.ws, it.number, kRowsTile, 0, D) : a.out;
    const long long to = SPLIT ? ((long long)row * D + half * HD) * 4 : ((long long)(it.start + col_k) * a.out_stride + elem) * (F32 ? 4 : 2);
    uint4 narrow[HD / 8];
#pragma unroll
    for (int c = 0; c < HD; c += 32) {  // 32 dims: a block
      float v[32];
      if constexpr (NP == 2) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[2 * j] = o[c / 2 + j].x, v[2 * j + 1] = o[c / 2 + j].y;
      } else {
        uint32_t r[32];
        if (nt > 0 && ok) {
          tmem_ld32(lanes + kColO + half * HD + c, r);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
      }
      const float factor = nan_blocks >> (c >> 5) & 1 ? NAN : inv;
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= factor;
      if constexpr (F32 || SPLIT) {
        uint4 own[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          own[j] = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
        rows_out<8>(turn, out, live ? to + c * 4 : -1, own);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          narrow[c / 8 + j] = make_uint4(as_u32(__floats2half2_rn(v[8 * j], v[8 * j + 1])), as_u32(__floats2half2_rn(v[8 * j + 2], v[8 * j + 3])),
                                         as_u32(__floats2half2_rn(v[8 * j + 4], v[8 * j + 5])), as_u32(__floats2half2_rn(v[8 * j + 6], v[8 * j + 7])));
      }
    }
    if constexpr (!F32 && !SPLIT) rows_out<HD / 8>(turn, out, live ? to : -1, narrow);
    tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && M.abort) *kv4_error_word(a.ws) = 1;
}

// ---------------- two row tiles per item ----------------
// Where K, V and the probabilities need one fp16 value each, an item is 256 rows: two tiles of 128 share every expanded
// K and V, and their softmaxes, four warps each with a whole row per thread, are independent, so one's chain of
// reads, maxima, exponentials and writes runs beside the other's.  P takes the place of its S in TMEM; the next
// scores that are written there wait for the product that reads P.  q lies in shared memory: TMEM holds the two tiles'
// S and P, two of each, and O.  The products' warp is the narrow place: each of its waits costs a hundred cycles though the
// barrier has long been passed, so K and V are waited for once per tile, not once per row tile (355 -> 343 us).
constexpr uint32_t kColPairS = 0, kColPairO = 256;

template <int D, int MODE>
__global__ void __launch_bounds__(kChunkThreads, 1) kv4_pair_kernel(const ChunkArgs a) {
  constexpr bool SPLIT = MODE == kParts;
  constexpr int KS = 3, q_tile = kRowsTile * D * 2;
  using L = ChunkLayout<D, 1, KS, 2 * q_tile>;
  extern __shared__ unsigned char chunk_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)chunk_raw + 1023) & ~(uintptr_t)1023);
  ChunkMisc& M = *reinterpret_cast<ChunkMisc*>(sm + L::off_misc);
  ChunkBars& B = M.bar;
  volatile int* abort_flag = &M.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ChunkItems<2 * kRowsTile, MODE> items(a);
  const ChunkItem& it = items.it;
  // the item's tiles of positions that its row tile g sees
  auto tiles_of = [&](int g) {
    const int r0 = it.row0 + g * kRowsTile;
    const int all = r0 < it.ncols ? (items.seen(min(it.ncols, r0 + kRowsTile) - 1) + kPosTile - 1) / kPosTile : 0;
    return min(max(all - it.t0, 0), it.nt);
  };

  if (tid == 0) chunk_init(M);
  if (warp == 0) {
    tmem_alloc(&M.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = M.tmem;

  if (warp >= kSoftWarps && warp < kSoftWarps + kProdWarps) {
    regs_down<kRegsProd>();
    chunk_expand<D, 1, 1, KS, L>(sm, M, items);
  } else if (warp >= kSoftWarps + kProdWarps) {
    regs_down<kRegsRest>();
    if (warp == kSoftWarps + kProdWarps + 1 && (MODE == kLoose || lane == 0) && !a.stall) chunk_copy<D, L>(sm, M, items);
    if (warp == kSoftWarps + kProdWarps) {
      // ---------------- products (as in the kernel with one row tile: one elected thread of a converged warp) ----------------
      const bool leader = elect_one();
      constexpr uint32_t id_s = idesc_f16_f32(kRowsTile, kPosTile), id_o = idesc_f16_f32(kRowsTile, D);
      const uint64_t qd = desc_sw128(smem_u32(sm)), kd = desc_sw128(smem_u32(sm + L::off_k)), vd = desc_sw128(smem_u32(sm + L::off_v));
      uint32_t s_count[2] = {0, 0}, o_count[2] = {0, 0}, q_ph[2] = {0, 0};  // of each row tile: scores and outputs so far
      // scores of row tile g and tile number ni; `last`: nobody reads this K after; `there`: it has been waited for
      auto scores = [&](int g, int ni, bool last, bool there) {
        const uint32_t c = s_count[g], b = c & 1, st = (uint32_t)ni % KS;
        bool ok = there || cwait(&B.k_full[st], (uint32_t)ni / KS & 1u, abort_flag);
        if (c >= 2) ok = ok && cwait(&B.pair_o[g][b], (c / 2 + 1) & 1u, abort_flag);  // the product that read this place's P
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc_fence_after();
        const uint64_t kb = kd + st * (uint32_t)(L::k_part >> 4), qb = qd + (uint32_t)g * (uint32_t)(q_tile >> 4);
        const uint32_t d = tmem + kColPairS + g * 128 + b * kPosTile;
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_bf16(d, qb + (((ks >> 2) * (kRowsTile * 128) + (ks & 3) * 32) >> 4),
                      kb + (((ks >> 2) * (kPosTile * 128) + (ks & 3) * 32) >> 4), id_s, ks ? 1u : 0u);
          if (last) umma_commit(&B.k_empty[st]);
          umma_commit(&B.pair_s[g][b]);
          mbar_arrive(&B.pair_s[g][b]);  // hands on what the producers wrote beside the tile
        }
        __syncwarp();
        ++s_count[g];
        return true;
      };
      // its output; `more`: added to the last tile's
      auto outputs = [&](int g, int ni, bool more, bool last, bool there) {
        const uint32_t c = o_count[g], b = c & 1, st = (uint32_t)ni % KS;
        const bool ok = (there || cwait(&B.v_full[st], (uint32_t)ni / KS & 1u, abort_flag)) && cwait(&B.pair_p[g][b], c / 2 & 1u, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc_fence_after();
        const uint64_t vb = vd + st * (uint32_t)(L::v_part >> 4);
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < kPosTile / 16; ++ks)
            umma_f16_ts(tmem + kColPairO + g * 128, tmem + kColPairS + g * 128 + b * kPosTile + ks * 8, vb + ((ks * 32) >> 4), id_o,
                        more || ks ? 1u : 0u);
          if (last) umma_commit(&B.v_empty[st]);
          umma_commit(&B.pair_o[g][b]);
          mbar_arrive(&B.pair_o[g][b]);
        }
        __syncwarp();
        ++o_count[g];
        return true;
      };
      bool ok = true;
      int n = 0;
      for (; ok && items.next(); n += it.nt) {
        const int nt0 = tiles_of(0), nt1 = tiles_of(1);
        for (int g = 0; g < 2; ++g)
          if (ok && (g ? nt1 : nt0) > 0) {
            ok = __all_sync(0xffffffffu, cwait(&B.pair_q[g], q_ph[g], abort_flag));
            q_ph[g] ^= 1;
          }
        if (!ok) break;
        tc_fence_after();
        if (nt0 > 0) ok = scores(0, n, nt1 <= 0, false);
        if (ok && nt1 > 0) ok = scores(1, n, true, nt0 > 0);
        if (ok && nt0 > 1) ok = scores(0, n + 1, nt1 <= 1, false);
        for (int i = 0; ok && i < it.nt; ++i) {
          if (i < nt0) ok = outputs(0, n + i, i > 0, i >= nt1, false);
          if (ok && i + 1 < nt1) ok = scores(1, n + i + 1, true, i + 1 < nt0);
          if (ok && i < nt1) ok = outputs(1, n + i, i > 0, true, i < nt0);
          if (ok && i + 2 < nt0) ok = scores(0, n + i + 2, i + 2 >= nt1, false);
        }
      }
      if (leader) {  // the products finish before TMEM is released, whoever has given up waiting for them
        umma_commit(&B.drain);
        mbar_wait(&B.drain, 0u, kDrainNs);
      }
    }
  } else {
    // ---------------- softmax ----------------
    regs_up<kRegsSoft>();
    const int g = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t place_s = lanes + kColPairS + g * 128, place_o = lanes + kColPairO + g * 128;
    bool ok = true;
    int n = 0;
    uint32_t c = 0;  // tiles of this row tile so far
    for (; items.next(); n += it.nt) {
      const int r0 = it.row0 + g * kRowsTile, nt = tiles_of(g);
      if (r0 >= it.ncols) continue;
      const int lim_lo = items.seen(r0), col = r0 + row, col_k = col / a.group;
      const bool live = col < it.ncols;
      const int lim = live ? items.seen(col) : 0;
      const long long elem = live ? (long long)(it.head * a.group + col - col_k * a.group) * D : 0;
      // ---- q into shared memory: fp16, scaled by a power of two per row, eight dims in the order of the unpacked codes
      // (0, 4, 1, 5, 2, 6, 3, 7).  The last item's scores are done with their q: this thread has waited for them
      float zscale;
      {
        uint4 raw[D / 8];
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                          (live ? (long long)(it.start + col_k) * a.q_stride + elem : 0));
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          raw[j] = live ? src[j] : make_uint4(0, 0, 0, 0);
          const uint32_t u[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u))));
        }
        const int e = top <= FLT_MAX ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 0;
        zscale = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(e - 13 + 127) << 23);
        const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
        unsigned char* tile = sm + g * q_tile;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const uint32_t u[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
          uint32_t h[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {  // dims t and t + 4
            const uint32_t lo = u[t >> 1], hi = u[2 + (t >> 1)];
            const float x0 = t & 1 ? __uint_as_float(lo & 0xffff0000u) : __uint_as_float(lo << 16);
            const float x1 = t & 1 ? __uint_as_float(hi & 0xffff0000u) : __uint_as_float(hi << 16);
            h[t] = as_u32(__floats2half2_rn(x0 * up, x1 * up));
          }
          *reinterpret_cast<uint4*>(tile + (j >> 3) * (kRowsTile * 128) + sw128_offset(row, 8 * (j & 7))) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_async_smem();
        if (nt > 0) mbar_arrive(&B.pair_q[g]);
      }

      float ref = -INFINITY, sum = 0.f;
      int nan_blocks = 0;  // the blocks of dims in which the row sees a V scale that is no number
      auto products_done = [&](uint32_t count) {  // of the row tile's tile number `count`
        if (!__all_sync(0xffffffffu, cwait(&B.pair_o[g][count & 1], count / 2 & 1u, abort_flag))) return false;
        tc_fence_after();
        return true;
      };
      auto note_bad = [&](int i) {
        if (M.bad[i & (kInfo - 1)]) {
#pragma unroll
          for (int b = 0; b < D / 32; ++b)
            if (M.first_bad[i & (kInfo - 1)][b] < lim) nan_blocks |= 1 << b;
        }
      };
      for (int i = 0; ok && i < nt;) {  // chains of tiles
      if (i > 0) {
        ok = products_done(c - 1);
        if (!ok) break;
        chain_sums<D, 2 * kRowsTile, D, true>(a.ws, SPLIT ? it.number : (long long)blockIdx.x, SPLIT ? a.count : (long long)gridDim.x, g * kRowsTile + row, 0, place_o, ref, i == kChain);
      }
      for (const int end = min(nt, i + kChain); i < end; ++i, ++c) {
        const int ni = n + i, inf = ni & (kInfo - 1);
        const uint32_t b = c & 1;
        ok = __all_sync(0xffffffffu, cwait(&B.pair_s[g][b], c / 2 & 1u, abort_flag));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[2][32];
        tmem_ld32(place_s + b * kPosTile, s[0]);
        tmem_ld32(place_s + b * kPosTile + 32, s[1]);
        float f = zscale;
        const float ev = M.v_exp[inf], v_inv = M.v_inv[inf];
        const int odd = M.odd[inf];
        if (i >= 2) note_bad(ni - 2);
        tmem_wait_ld();
        const int pos0 = (it.t0 + i) * kPosTile;
        if (pos0 + kPosTile > lim_lo || odd) {
          if (odd & kWide) {
#pragma unroll
            for (int j = 0; j < kPosTile; ++j)
              s[j >> 5][j & 31] = __float_as_uint(__uint_as_float(s[j >> 5][j & 31]) * M.k_pos_pow[inf][j]);
          }
          if (odd & kSpread) {
#pragma unroll
            for (int j = 0; j < kPosTile; ++j)
              s[j >> 5][j & 31] = __float_as_uint(fmaf(__uint_as_float(s[j >> 5][j & 31]), f, M.v_pos_exp[inf][j]));
            f = 1.f;
          }
#pragma unroll
          for (int j = 0; j < kPosTile; ++j)
            if (pos0 + j >= lim || (odd >> (j >> 4) & 1)) s[j >> 5][j & 31] = 0xff800000u;
        }
        float m4[4];  // four chains
#pragma unroll
        for (int j = 0; j < 4; ++j) m4[j] = __uint_as_float(s[0][j]);
#pragma unroll
        for (int j = 4; j < kPosTile; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(s[j >> 5][j & 31]));
        const float most = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), f, ev);
        float keep = 1.f;
        if (most - kChunkTop<1> > ref + kChunkSlack<1>) {
          keep = exp2_approx(ref - (most - kChunkTop<1>));
          ref = most - kChunkTop<1>;
          sum *= keep;
        }
        const float base = ev - (ref == -INFINITY ? 0.f : ref);
        const bool moved = __any_sync(0xffffffffu, keep != 1.f) && i > 0;
        if (moved || (odd & kSpread)) {
          if (odd & kSpread) {  // the sum by each position's power; the one below counts for 0 (v_inv)
#pragma unroll
            for (int j = 0; j < kPosTile; ++j) sum += exp2_approx(__uint_as_float(s[j >> 5][j & 31]) - M.v_pos_exp[inf][j] + base);
          }
          if (moved) {
            ok = products_done(c - 1);
            if (!ok) break;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
              uint32_t r[16];
              tmem_ld16(place_o + d, r);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * keep);
              tmem_st16(place_o + d, r);
            }
          }
        }
        float2 part4[4];  // four chains
#pragma unroll
        for (int j = 0; j < 4; ++j) part4[j] = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t hi[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 z = fma2(make_float2(__uint_as_float(s[h][2 * j]), __uint_as_float(s[h][2 * j + 1])), make_float2(f, f), make_float2(base, base));
            const float2 x = make_float2(exp2_approx(z.x), exp2_approx(z.y));
            part4[j & 3] = add2(part4[j & 3], x);
            hi[j] = as_u32(__floats2half2_rn(x.x, x.y));
          }
          tmem_st16(place_s + b * kPosTile + 16 * h, hi);  // over the thread's own scores, which are read
        }
        const float2 part = add2(add2(part4[0], part4[1]), add2(part4[2], part4[3]));
        sum = fmaf(part.x + part.y, v_inv, sum);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&B.pair_p[g][b]);
      }
      }
      if (ok && nt > 0) {
        ok = products_done(c - 1);
        if (ok && nt > kChain) chain_sums<D, 2 * kRowsTile, D, false>(a.ws, SPLIT ? it.number : (long long)blockIdx.x, SPLIT ? a.count : (long long)gridDim.x, g * kRowsTile + row, 0, place_o, ref, false);
        if (nt > 1) note_bad(n + nt - 2);
        note_bad(n + nt - 1);
      }
      const float inv = !ok ? NAN : SPLIT ? 1.f : sum != 0.f ? 1.f / sum : 0.f;  // rows that could not be finished are NaN
      if (SPLIT) *part_ml(a.ws, a.count, it.number, 2 * kRowsTile, g * kRowsTile + row, D) = make_float2(ref, sum);
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {  // a block of dims
        uint32_t r[32];
        if (ok && nt > 0) {
          tmem_ld32(place_o + d, r);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0;
        }
        const float factor = nan_blocks >> (d >> 5) & 1 ? NAN : inv;
        if (live && SPLIT) {
          float4* out = reinterpret_cast<float4*>(part_row(a.ws, it.number, 2 * kRowsTile, g * kRowsTile + row, D) + d);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            out[j] = make_float4(__uint_as_float(r[4 * j]) * factor, __uint_as_float(r[4 * j + 1]) * factor,
                                 __uint_as_float(r[4 * j + 2]) * factor, __uint_as_float(r[4 * j + 3]) * factor);
        } else if (live) {
          uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + (long long)(it.start + col_k) * a.out_stride + elem + d);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[8 * j + 2 * k]) * factor, __uint_as_float(r[8 * j + 2 * k + 1]) * factor);
              u[k] = *reinterpret_cast<const uint32_t*>(&v);
            }
            out[j] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
        __syncwarp();  // the next block's TMEM read is the whole warp's
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && M.abort) *kv4_error_word(a.ws) = 1;
}

// Joins the parts of a row, in their order: a warp per row.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) kv4_join_kernel(const ChunkArgs a, int dtype) {
  constexpr int rows = ROWS;
  constexpr int N = D / 32;  // dims of a lane
  const int parts = a.parts;
  ChunkItems<ROWS, kParts> items(a);
  const ChunkItem& it = items.it;
  const long long first = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);  // row, counted over all row tiles
  const int lane = threadIdx.x & 31, row = (int)(first % rows);
  const long long number = first / rows * parts;
  if (number >= a.count || !items.at(number) || it.row0 + row >= it.ncols) return;
  float top = -INFINITY, sum = 0.f, v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int p = 0; p < parts; ++p) top = fmaxf(top, part_ml(a.ws, a.count, number + p, rows, row, D)->x);
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float2 ml = *part_ml(a.ws, a.count, number + p, rows, row, D);
    const float k = ml.x == top ? 1.f : exp2_approx(ml.x - top);
    const float* src = part_row(a.ws, number + p, rows, row, D) + lane * N;
    sum = fmaf(ml.y, k, sum);
    if constexpr (N == 4) {
      const float4 x = *reinterpret_cast<const float4*>(src);
      v[0] = fmaf(x.x, k, v[0]), v[1] = fmaf(x.y, k, v[1]), v[2] = fmaf(x.z, k, v[2]), v[3] = fmaf(x.w, k, v[3]);
    } else {
      const float2 x = *reinterpret_cast<const float2*>(src);
      v[0] = fmaf(x.x, k, v[0]), v[1] = fmaf(x.y, k, v[1]);
    }
  }
  const int at = it.row0 + row, k = at / a.group;
  const long long out = (long long)(it.start + k) * a.out_stride + (it.head * a.group + at % a.group) * D + lane * N;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) store_elem(a.out, dtype, out + i, v[i] * inv);
}

// Where the row tiles alone leave SMs without work, the positions of each are shared out over `parts` items, of four
// tiles at least (one sequence of 32768 positions, 8 KV heads: 64 rows each in STAGE_F32 66 us, 858 in one part; 256 in
// STAGE_BF16 74 us, 748 in one).
int chunk_parts(long long row_tiles, int max_len, int sms) {
  const long long tiles = (max_len + kPosTile - 1) / kPosTile;
  const long long most = min((long long)min(sms, kKv4ChunkParts) / max(row_tiles, 1ll), tiles / 4);
  return (int)max(1ll, most);
}

// Launches a kernel, one CTA per SM at most.
template <typename Kernel>
cudaError_t launch_items(Kernel* kern, int smem, const ChunkArgs& a, std::atomic<uint64_t>& ready, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {  // once per device
    // The warpgroups share out kRegsStart registers a thread: from a compiler that gave the kernel fewer, the one that asks for more
    // would wait forever
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < kRegsStart) return cudaErrorLaunchOutOfResources;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  // the workspace has places for kKv4ChunkParts CTAs' chains
  kern<<<(int)min(a.count, (long long)min(sm_count(), kKv4ChunkParts)), kChunkThreads, smem, st>>>(a);
  return cudaGetLastError();
}

// The kernel for one row tile per item, or (PAIR) for two.
template <int D, int NQ, int NKV, int NP, bool PAIR, int MODE>
cudaError_t launch_mode(const ChunkArgs& a, int dtype, cudaStream_t st) {
  constexpr int ROWS = (PAIR ? 2 : 1) * kRowsTile;
  constexpr int smem = PAIR ? ChunkLayout<D, 1, 3, 2 * kRowsTile * D * 2>::bytes : ChunkLayout<D, NKV, 2, kSoftWarps * kTurn>::bytes;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  static std::atomic<uint64_t> ready{0};
  cudaError_t e;
  if constexpr (PAIR) e = launch_items(kv4_pair_kernel<D, MODE>, smem, a, ready, st);
  else e = launch_items(kv4_chunk_kernel<D, NQ, NKV, NP, MODE>, smem, a, ready, st);
  if (MODE != kParts || e != cudaSuccess) return e;
  kv4_join_kernel<D, ROWS><<<(unsigned)((a.count / a.parts * ROWS + 7) / 8), 256, 0, st>>>(a, dtype);
  return cudaGetLastError();
}

thread_local int g_stalls = 0;  // calls of this thread still to be stalled

template <int D, int NQ, int NKV, int NP, bool PAIR>
cudaError_t launch_chunk(const Kv4AttnArgs& args, int dtype, cudaStream_t st) {
  constexpr int ROWS = (PAIR ? 2 : 1) * kRowsTile;
  ChunkArgs a;
  static_cast<Kv4AttnArgs&>(a) = args;
  a.group = a.n_q_heads / a.c.n_kv_heads;
  a.row_tiles = (int)(((long long)a.max_q * a.group + ROWS - 1) / ROWS);
  const long long tiles = (long long)a.row_tiles * a.c.n_kv_heads * a.n_seqs;
  a.parts = chunk_parts(tiles, a.max_len, sm_count());
  a.count = tiles * a.parts;
  a.stall = g_stalls > 0 ? g_stalls-- > 0 : 0;
  if (a.parts > 1) return launch_mode<D, NQ, NKV, NP, PAIR, kParts>(a, dtype, st);
  // no more items than this, however the tokens are spread over the sequences
  const long long items = ((long long)a.n_tok * a.group / ROWS + a.n_seqs) * a.c.n_kv_heads;
  return tiles > 2 * items ? launch_mode<D, NQ, NKV, NP, PAIR, kLoose>(a, dtype, st) : launch_mode<D, NQ, NKV, NP, PAIR, kTight>(a, dtype, st);
}

}  // namespace

void kv4_stall(int calls) { g_stalls = calls; }

size_t kv4_chunk_ws_bytes(int head_dim) {
  return kKv4CounterBytes + (size_t)kKv4ChunkParts * 2 * kRowsTile * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv4_chunk(const Kv4AttnArgs& a, int head_dim, int dtype, cudaStream_t st) {
  if (head_dim == 128) {
    if (dtype == KV4_F32) return launch_chunk<128, 2, 2, 2, false>(a, dtype, st);
    if (dtype == KV4_F16) return launch_chunk<128, 1, 2, 1, false>(a, dtype, st);
    return launch_chunk<128, 1, 1, 1, true>(a, dtype, st);
  }
  if (dtype == KV4_F32) return launch_chunk<64, 2, 2, 2, false>(a, dtype, st);
  if (dtype == KV4_F16) return launch_chunk<64, 1, 2, 1, false>(a, dtype, st);
  return launch_chunk<64, 1, 1, 1, true>(a, dtype, st);
}

}  // namespace lrs
