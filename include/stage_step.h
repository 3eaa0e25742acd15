/*
 * layer_range_stage (GB300) -- a step's operators around the projections.
 *
 * What a program that puts a decoder's step together from single ops needs between the residual
 * stream and the paged cache (stage_kv4.h), and behind the logits; in the manner of stage_ops.h
 * (return codes of stage.h, messages through stage_op_last_error(), no C++ exception crosses the
 * boundary, nothing is allocated or synchronised):
 *
 *   stage_op_norm_f8    the residual's addition, an RMS norm, and rows of 8 bits with their scales
 *   stage_op_f8_gemm    rows of 8 bits times a weight matrix of 8 bits, a scale for each block of 128
 *   stage_op_rope       rotary positions of query and key heads
 *   stage_op_logprobs   log probabilities of given tokens, entropy, ranks and the likeliest tokens
 *
 * 8-bit values are e4m3 (4 exponent bits, 3 of mantissa, largest 448, no infinities).  A matrix of
 * them has a float32 scale per block: a row of activations one per 128 columns, weights one per
 * 128 rows x 128 columns; a value is code * scale.
 */
#ifndef LAYER_RANGE_STAGE_STEP_H
#define LAYER_RANGE_STAGE_STEP_H

#include "stage_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The residual's addition, an RMS norm, and 8-bit rows with scales, for n_tok rows of n columns:
 *   h = x + resid                  rounded to float32, then to resid's type; written to resid_out
 *   h = x                          where resid_dev is NULL (resid_out_dev is NULL too)
 *   y = (h * r) * gamma            each product rounded to float32, with r = 1 / sqrt(mean(h^2) + eps) rounded once
 *   y = h                          where gamma_dev is NULL (rows that are quantised as they are)
 *   per block of 128 columns:      a = max(largest |y|, 2^-100), scale = a / 448, code = e4m3(y * (448 / a))
 * with every quotient and product rounded to nearest in float32 and the code to nearest, ties to even: the same
 * codes on any machine.  (r is the float32 next to the exact one but for one row in about a million, where it
 * may be the neighbour.)
 *   x_dev: [n_tok] rows of x_dtype at x_stride elements; resid_dev, resid_out_dev: rows of resid_dtype, which is
 *     x_dtype or STAGE_F32; resid_out_dev may be resid_dev, with the same stride.
 *   gamma_dev: float32 [n]; eps >= 0.
 *   q_dev: codes, [n_tok] rows at q_stride bytes; scale_dev: float32 [ceil(n / 128)] rows of n_tok at scale_stride
 *     elements (block after block, as stage_op_f8_gemm reads them).  Both may be NULL when y_dev is given.
 *   y_dev: y rounded once to x_dtype, rows at y_stride elements, or NULL.
 * Bytes between a row's n columns and the next row are left as they were.  A row whose sum of squares is no finite
 * float32, or whose mean + eps is below 2^-256 (zeros with eps = 0), gives NaN throughout (with gamma); a block that holds an
 * infinity or a NaN gets a scale that is not finite: all of it reads as NaN.  Apart from resid_out = resid no output may overlap
 * an input or another output.
 * Rows need their elements' alignment only; with rows and bases at multiples of four elements they are read and written four
 * elements at a time.  Runs on `stream`.  n_tok = 0 does nothing.  Errors: STAGE_E_INVALID (null or unaligned
 * pointers, types, n_tok outside [0, 2^24], n outside [1, 32768], strides below a row or above 2^32, eps negative
 * or not finite), STAGE_E_CUDA (the launch). */
STAGE_API int stage_op_norm_f8(const void* x_dev, int x_dtype, int64_t x_stride, const void* resid_dev, int resid_dtype,
                               int64_t resid_stride, void* resid_out_dev, int64_t resid_out_stride,
                               const float* gamma_dev, float eps, int n_tok, int n, void* q_dev, int64_t q_stride,
                               float* scale_dev, int64_t scale_stride, void* y_dev, int64_t y_stride, void* stream);

/* y[m][r] = sum_b a_scale[b][m] * w_scale[r / 128][b] * sum_{k in block b} a[m][k] * w[r][k], for m < M, r < N,
 * with blocks of 128 along K (the last may be shorter).
 *   a_dev: e4m3 codes, M rows of K at a_stride bytes; a_scale_dev: float32 [ceil(K / 128)] rows of M at a_scale_stride
 *     elements (stage_op_norm_f8 writes both).
 *   w_dev: e4m3 codes, N rows of K at w_stride bytes; w_scale_dev: float32 [ceil(N / 128)][ceil(K / 128)], contiguous.
 *   y_dev: rows of y_dtype at y_stride elements, rounded once; it overlaps no input.
 *   error_dev: device int32 or NULL, set to 1 where the GPU did not finish a copy or a product within a second; what misses
 *     it is NaN.  No call clears it.
 * a_dev, w_dev and both row strides must be multiples of 16 bytes (what lies between a row's K codes and the next row does not
 * matter); y needs its elements' alignment, and is written 16 bytes at a time where base and rows are multiples of that.
 * Sums of a block are the tensor cores' float32, sums over blocks float32 in a fixed order: the same inputs give the same
 * bits for the same M.  The two scales are multiplied first, in float32: where their product is below 2^-126 it loses bits, and
 * where it is infinite so is what it scales, or NaN.
 * Runs on `stream`.  M = 0 does nothing.  Errors: STAGE_E_INVALID (null or unaligned pointers, type, M outside
 * [0, 2^24], N outside [1, 2^24], M * N above 2^40, K outside [1, 2^20], strides below a row, not a multiple of 16 bytes (a, w) or above
 * 2^32), STAGE_E_CUDA (tensor maps or the launch). */
STAGE_API int stage_op_f8_gemm(const void* a_dev, int64_t a_stride, const float* a_scale_dev, int64_t a_scale_stride,
                               const void* w_dev, int64_t w_stride, const float* w_scale_dev, int M, int N, int K,
                               void* y_dev, int y_dtype, int64_t y_stride, int32_t* error_dev, void* stream);

/* For tests: the next `calls` calls of stage_op_f8_gemm by this thread copy nothing, so that their waits run out: everything is
 * NaN and the error word is set.  Nothing faults, traps or hangs.  calls = 0 takes it back.  Host only.  Errors:
 * STAGE_E_INVALID (calls outside [0, 16]). */
STAGE_API int stage_op_f8_debug_stall(int calls);

/* For tests: in the next `calls` calls of stage_op_f8_gemm by this thread one warp of each SM gives up on its second tile of 256 x 256,
 * as if the product had come just too late (M above 128 and more such tiles than there are pairs of SMs; other calls are as ever).
 * What it misses is NaN, everything else right, and the error word is set.  calls = 0 takes it back.  Host only.  Errors:
 * STAGE_E_INVALID (calls outside [0, 16]). */
STAGE_API int stage_op_f8_debug_late(int calls);

/* How the frequencies of rotary positions are scaled for contexts `factor` times as long as first_len. */
enum {
  STAGE_ROPE_PLAIN = 0,  /* f_i = theta^(-2 i / rot_dim) */
  STAGE_ROPE_LINEAR = 1, /* f_i / factor */
  STAGE_ROPE_BASE = 2,   /* theta * factor^(rot_dim / (rot_dim - 2)) in theta's place */
  STAGE_ROPE_BANDS = 3,  /* f_i / factor where first_len holds fewer than `low` of its waves, f_i where more than `high`, mixed
                            linearly in their number between */
  STAGE_ROPE_PARTS = 4   /* the same by the pair's index, linearly from the (rounded down) index at which first_len holds `high`
                            waves to the (rounded up) one at which it holds `low`; scale = 0.1 ln(factor) + 1 */
};

/* Frequencies (radians per position, rot_dim / 2 float64 on the host) and the factor `scale` of stage_op_rope
 * (1 but for STAGE_ROPE_PARTS).  first_len, low and high matter for BANDS and PARTS only.  Host only.  Errors:
 * STAGE_E_INVALID (null pointers; rot_dim odd or outside [2, 1024], 2 for BASE; theta <= 1; a factor below 1; first_len < 1; low
 * <= 0 or high <= low; an unknown scaling). */
STAGE_API int stage_op_rope_freqs(int rot_dim, double theta, int scaling, double factor, double first_len, double low,
                                  double high, double* freqs, float* scale);

/* Rotary positions: in every head of a token's q and k, the pair (u, v) number i < rot_dim / 2 becomes
 *   (u cos a - v sin a, v cos a + u sin a) * scale,    a = pos * freqs[i],
 * where pair i is dims (2 i, 2 i + 1) if `interleaved`, else (i, i + rot_dim / 2); dims from rot_dim on are unchanged.
 *   q_dev: [n_tok] rows of n_q_heads * head_dim elements of `dtype` at q_stride elements; k_dev the same with n_k_heads, or NULL with
 *     n_k_heads = 0; q and k may be parts of one fused row.
 *   q_out_dev, k_out_dev: rows of the same form; each may be its input, with the same stride, and else overlaps
 *     nothing.
 *   pos_dev: device int32 [n_tok]; a token whose pos is negative is padding: its output rows are left as they were
 *     (stage_op_kv4_plan writes pos like this).
 *   freqs_dev: device float64 [rot_dim / 2], radians per position, finite.  Angles are taken as 64-bit fractions of a turn, so that they
 *     are as good as freqs at any position; cos, sin and the rotation are float32, rounded once to dtype.
 * Rows need their elements' alignment; where bases, strides, head_dim and rot_dim allow it they are read and written 16 bytes
 * at a time.  Runs on `stream`.  n_tok = 0 does nothing.  Errors: STAGE_E_INVALID (null or unaligned pointers, dtype,
 * n_tok outside [0, 2^24], n_q_heads outside [1, 1024], n_k_heads outside [0, 1024], head_dim outside [2, 1024], rot_dim
 * odd or outside [2, head_dim], strides below a row or above 2^32, a scale that is not finite), STAGE_E_CUDA (the launch). */
STAGE_API int stage_op_rope(const void* q_dev, int64_t q_stride, int n_q_heads, const void* k_dev, int64_t k_stride,
                            int n_k_heads, int head_dim, int dtype, const int32_t* pos_dev, int n_tok,
                            const double* freqs_dev, int rot_dim, int interleaved, float scale, void* q_out_dev,
                            int64_t q_out_stride, void* k_out_dev, int64_t k_out_stride, void* stream);

#define STAGE_LOGPROBS_MAX_TOP 32

/* Log probabilities from logits: for each of n_rows rows z of `vocab` logits, with p = softmax(z),
 *   logprob = log p[t] of the given token t, entropy = -sum p log p (in nats; a logit of -inf adds nothing),
 *   rank = the number of tokens before t in the order of falling logits, equal ones by their index (0: the likeliest),
 *   top_ids, top_logprobs = the n_top first tokens of that order and their log p.
 *   logits_dev: rows of `dtype` at row_stride elements (elements' alignment is enough); -inf, and a type's lowest value, mask a
 *     token.  Arithmetic is float32.
 *   tokens_dev: device int32 [n_rows]; a token outside [0, vocab) gets a logprob of NaN and a rank of -1 (nothing else of
 *     its row changes).  NULL: logprob_dev and rank_dev are NULL too.
 *   logprob_dev [n_rows], entropy_dev [n_rows]: float32; rank_dev [n_rows]: int32; top_ids_dev int32 and top_logprobs_dev
 *     float32 [n_rows][n_top].  Each may be NULL; n_top = 0 has no top (at most STAGE_LOGPROBS_MAX_TOP, and vocab).
 * A row that holds a NaN or +inf, or nothing but -inf, has no distribution: its logprob, entropy and top_logprobs are NaN, its rank
 * and top_ids -1.  The same inputs give the same bits.  Runs on `stream`.  n_rows = 0 does nothing.  Errors:
 * STAGE_E_INVALID (null or unaligned pointers, dtype, n_rows outside [0, 2^24], vocab outside [1, 2^19], row_stride below vocab or
 * above 2^32, n_top), STAGE_E_CUDA (the launch). */
STAGE_API int stage_op_logprobs(const void* logits_dev, int dtype, int64_t row_stride, int n_rows, int vocab,
                                const int32_t* tokens_dev, float* logprob_dev, float* entropy_dev, int32_t* rank_dev,
                                int n_top, int32_t* top_ids_dev, float* top_logprobs_dev, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LAYER_RANGE_STAGE_STEP_H */
