/*
 * layer_range_stage (GB300) -- a paged KV cache held in 4 bits.
 *
 * Operators of a batched decoding stage, on caller-owned device buffers, in the manner of
 * stage_ops.h (return codes of stage.h, messages through stage_op_last_error(), no C++
 * exception crosses the boundary, nothing is allocated or synchronised):
 *
 *   stage_op_kv4_plan       block tables and slot maps built on the GPU from request lengths
 *   stage_op_kv4_append     K and V rows quantised to 4 bits and written to their slots
 *   stage_op_kv4_read       the rows at some slots as values
 *   stage_op_kv4_attention  softmax(q k^T / sqrt(head_dim)) v over the pages, causal
 *
 * One step of a serving loop calls plan, then per block append and attention; every length
 * and index they go by is on the device, so the step can be captured in a CUDA graph and
 * replayed while the sequences grow.
 *
 * The cache is one device buffer of stage_op_kv4_cache_bytes(...) bytes:
 *   [page][kv head][tile of 16 positions][bytes of a tile]
 * with page_len positions per page (a multiple of 16, at most 4096).  A tile holds, in this order,
 *   K codes   [position 16][dim / 8 % 4][block][4 bytes]   byte dim / 2 % 4, low nibble = lower dim
 *   K scales  [position 16][block] fp16
 *   V codes   [position / 8][dim / 4 % 8][position / 2 % 4][position % 2][block][2 bytes]
 *                                                           byte dim / 2 % 2, low nibble = lower dim
 *   V scales  [position 16][block] fp16
 * where a block is 32 neighbouring dims (block = dim / 32): 18 * head_dim bytes per tile, 4.5 bits
 * per value.  The codes are ordered so that one 16-byte load gives a lane of the attention kernel
 * its operands of the tensor-core product; every byte belongs to one position.  A code c
 * stands for s * (c - 8), exactly, with its block's scale s.
 *
 * A slot is the place of one position in the cache: page * page_len + offset.  head_dim is 64
 * or 128.  n_pages * page_len is at most 2^31 - 1; byte offsets are 64-bit throughout.
 */
#ifndef LAYER_RANGE_STAGE_KV4_H
#define LAYER_RANGE_STAGE_KV4_H

#include "stage_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of the rows that append, read and attention take and give. */
enum { STAGE_F32 = 0, STAGE_F16 = 1, STAGE_BF16 = 2 };

/* What stage_op_kv4_plan writes to its status word. */
enum {
  STAGE_PLAN_OK = 0,
  STAGE_PLAN_NO_PAGES = 1, /* the requests need more pages than are free */
  STAGE_PLAN_BAD_LEN = 2,  /* a length that is negative, a kept length above the cached one, a request beyond
                              its table row or 2^31 - 1 positions, or a ring whose state does not fit its size */
  STAGE_PLAN_NO_ROOM = 3   /* more new tokens than the slot map holds */
};

/* Bytes of a cache (0 for sizes that no call accepts). */
STAGE_API size_t stage_op_kv4_cache_bytes(int64_t n_pages, int page_len, int n_kv_heads, int head_dim);

/* Block tables and slot maps of one step, from the lengths of its requests.
 *
 * Request i has seq_len[i] positions in the cache, of which keep_len[i] stay (NULL: all of them;
 * fewer when a draft is rolled back; 0 when it has finished) and new_len[i] are added.  Its pages are the
 * first ceil(seq_len[i] / page_len) entries of its row of `table` [n_seqs][table_stride].  Where it
 * needs more pages afterwards they are taken from the free ring, request after request, and written to
 * its row; where it needs fewer, those behind go back to the ring's end and can be taken from the
 * next call on.  Table entries behind a request's pages are left as they were.
 *   free_ring [ring_len]: page ids; free_state[2] = (head, count): the free pages are
 *     free_ring[(head + j) % ring_len], j < count.  Pages are taken from the head.
 *   seq_len_out [n_seqs]: keep + new; may be seq_len.  free_state_out[2]: may be free_state.
 *   cu_new [n_seqs + 1]: prefix sums of new_len, from 0.
 *   slot, pos, seq [n_tok]: for token t of the step -- the k-th new token of request i, t = cu_new[i] + k --
 *     its slot, its position keep + k and i; -1 in all three behind the last token (and a
 *     slot of -1 where the table holds no page id from 0 to n_pages - 1).
 *   status [1]: STAGE_PLAN_*.  Where it is not STAGE_PLAN_OK the step is refused as a whole:
 *     seq_len_out and free_state_out repeat the inputs, cu_new is all 0, slot, pos and seq are
 *     all -1 -- append and attention then do nothing -- and table and ring are untouched.
 * Except for the two named pairs no output may overlap an input or another output.  Device int32
 * throughout.  One launch on `stream`.  Errors: STAGE_E_INVALID (null pointers; n_seqs outside
 * [0, 65536]; page_len; table_stride outside [1, 2^20]; n_pages, or n_pages * page_len, outside [1, 2^31);
 * ring_len outside [1, 2^30]; n_tok outside [0, 2^24]), STAGE_E_CUDA. */
STAGE_API int stage_op_kv4_plan(int n_seqs, int page_len, int64_t n_pages, const int32_t* seq_len_dev,
                                const int32_t* keep_len_dev, const int32_t* new_len_dev, int32_t* table_dev,
                                int table_stride, int32_t* free_ring_dev, int ring_len,
                                const int32_t* free_state_dev, int32_t* seq_len_out_dev, int32_t* free_state_out_dev,
                                int n_tok, int32_t* cu_new_dev, int32_t* slot_dev, int32_t* pos_dev, int32_t* seq_dev,
                                int32_t* status_dev, void* stream);

/* Quantise and write K and V rows.  k_dev, v_dev: [n_tok] rows of n_kv_heads * head_dim elements of
 * `dtype`, row t at t * row_stride elements (row_stride a multiple of 16 bytes, so that rows inside
 * a fused QKV output can be given).  slot_dev: device int32 [n_tok]; a row whose slot is outside
 * [0, n_pages * page_len) is skipped (padding); two rows with the same slot leave that slot undefined.
 * Per block of 32 dims: m = the element of largest magnitude (the lowest index of several), s = m / -8 rounded
 * to fp16, c = x / s rounded to the nearest integer (ties to even), plus 8, clamped to [0, 15]; x / s is
 * decided exactly.  s = 0 gives values of 0.  A block whose scale is not finite (an infinity, a NaN, or
 * a magnitude from 524160 on) gets the scale NaN: it reads as NaN.
 * Bytes of other positions are left as they were.  Runs on `stream`.  n_tok = 0 does nothing.  Errors:
 * STAGE_E_INVALID (null or unaligned pointers, cache sizes, dtype, row_stride, n_tok outside
 * [0, 2^24]), STAGE_E_CUDA (the launch). */
STAGE_API int stage_op_kv4_append(void* cache_dev, int64_t n_pages, int page_len, int n_kv_heads, int head_dim,
                                  const void* k_dev, const void* v_dev, int dtype, int64_t row_stride,
                                  const int32_t* slot_dev, int n_tok, void* stream);

/* The rows at n_tok slots as values: s * (c - 8), exact in STAGE_F32, rounded once to nearest
 * otherwise.  k_out_dev, v_out_dev: rows as in stage_op_kv4_append.  Rows whose slot is outside
 * [0, n_pages * page_len) are left as they were; the same slot may be read several times.  Errors as for
 * stage_op_kv4_append. */
STAGE_API int stage_op_kv4_read(const void* cache_dev, int64_t n_pages, int page_len, int n_kv_heads, int head_dim,
                                const int32_t* slot_dev, int n_tok, void* k_out_dev, void* v_out_dev, int dtype,
                                int64_t row_stride, void* stream);

/* Scratch bytes of stage_op_kv4_attention for these sizes (0 for sizes that no call accepts).  It
 * grows with the sizes, except that it never passes STAGE_KV4_SCRATCH_MAX. */
STAGE_API size_t stage_op_kv4_attention_workspace_bytes(int n_seqs, int n_q_heads, int n_kv_heads, int head_dim,
                                                        int max_q, int max_len);
#define STAGE_KV4_SCRATCH_MAX (64u << 20)
#define STAGE_KV4_ERROR_AT 2048

/* Which kernel a call of stage_op_kv4_attention with these sizes runs on: 1, the one for many columns (query tokens of a
 * sequence times query heads per KV head; a chunk of a prompt), whose precision is stated below as that of chunks; 0, the one
 * for few.  It goes by the bounds alone.  Host only.  Errors: STAGE_E_INVALID (sizes that no call accepts). */
STAGE_API int stage_op_kv4_attention_many(int n_seqs, int n_tok, int n_q_heads, int n_kv_heads, int head_dim, int dtype, int max_q,
                                          int max_len);

/* Attention over the paged 4-bit cache.
 *   q_dev: [n_tok] rows of n_q_heads * head_dim elements of `dtype` (already rotated), row t at
 *     t * q_stride elements; out_dev the same with out_stride (it may be q_dev, with the same stride, and else
 *     overlaps no input).  Query head j reads KV head
 *     j / (n_q_heads / n_kv_heads); any ratio.
 *   cu_q_dev [n_seqs + 1]: sequence i has the query tokens cu_q[i] .. cu_q[i + 1] - 1, not decreasing, at most n_tok;
 *   seq_len_dev [n_seqs]: its positions in the cache, those of its query tokens included: with
 *     c = cu_q[i + 1] - cu_q[i], query token k is position seq_len[i] - c + k and attends to the
 *     positions from 0 to that one (one token per sequence: decode; more: a chunk of a prompt, or
 *     drafts to be verified).
 *   table_dev [n_seqs][table_stride]: the pages, as stage_op_kv4_plan writes them.
 *   max_q, max_len: bounds of the query tokens of one sequence and of seq_len (host values, which decide the
 *     launch; with a captured graph, the bounds over its replays).  Tokens behind the max_q-th of a
 *     sequence get no output, and seq_len counts as at most max_len and table_stride * page_len.
 *   out: sum_j p_j v_j with p = softmax(q k^T / sqrt(head_dim)); a token with no position gets zeros.
 *     Rows behind cu_q[n_seqs] are left as they were.  Positions whose table entry is no page id count as absent;
 *     what the cache holds behind seq_len never matters.
 *     A scale that is no finite number (append writes NaN; another writer may leave infinities, which count as NaN): in K it
 *     makes NaN of the KV head's outputs of every token that sees the position, in V of its own block of dims in them.
 *   Arithmetic: sums, maxima and the softmax are float32.  STAGE_F32: q and the probabilities are each
 *     held as two fp16 values (22 bits) and meet exact integers or exact values, for an error of the
 *     order of float32's; what lies 2^34 or more below a row's largest p_j v_j counts as 0.  The 16-bit types round out
 *     once to nearest, and a probability may be rounded once to fp16; what lies 2^27 or more below a row's largest p_j v_j
 *     counts as 0.  STAGE_BF16 may also round K and V once to fp16 (11 bits, where the output has 8).  In all types an
 *     element of q 2^34 or more below its row's largest counts as 0 (and from 2^27 below on has fewer bits), and where a
 *     position's largest scale in K or V is 4096 or more, its values may be off by 2^-33 of its largest.  What a token
 *     does not see has no part in any of this.
 *     Where the GPU does not finish a copy or a product of a chunk within a second, the rows that miss it are NaN, and the
 *     32-bit word STAGE_KV4_ERROR_AT bytes into the workspace is set to 1; no call clears it (it is read, and cleared, where
 *     results are read: nothing here synchronises).
 *   workspace_dev: stage_op_kv4_attention_workspace_bytes(...) bytes whose contents must be zero
 *     before the first call (each call leaves it ready for the next, of any sizes it is large enough
 *     for); two calls that may run at the
 *     same time (on two streams, or in two graphs) need one each.
 * Every sum has a fixed order: the same inputs give the same bits.  Runs on `stream`.  n_seqs = 0 or
 * n_tok = 0 does nothing.  Errors: STAGE_E_INVALID (null or unaligned pointers, cache sizes, dtype, strides below
 * a row or not a multiple of 16 bytes, n_seqs outside [0, 65535], n_tok outside [0, 2^24], n_q_heads no
 * multiple of n_kv_heads or above 1024, max_q outside [1, 2^20], max_len outside [1, 2^30], table_stride outside
 * [1, 2^20], a workspace too small), STAGE_E_CUDA (the launch). */
STAGE_API int stage_op_kv4_attention(const void* cache_dev, int64_t n_pages, int page_len, int n_kv_heads,
                                     int head_dim, const void* q_dev, int dtype, int64_t q_stride, int n_tok,
                                     int n_q_heads, const int32_t* cu_q_dev, const int32_t* seq_len_dev,
                                     const int32_t* table_dev, int table_stride, int n_seqs, int max_q, int max_len,
                                     void* out_dev, int64_t out_stride, void* workspace_dev, size_t workspace_bytes,
                                     void* stream);

/* For tests: the next `calls` calls of stage_op_kv4_attention by this thread that run on the kernel for many columns copy
 * nothing of the cache, so that the waits for it run out: every row is NaN, the error word is set, and the workspace is ready for
 * the next call.  Nothing faults, traps or hangs.  calls = 0 takes it back.  Host only.  Errors: STAGE_E_INVALID (calls outside
 * [0, 16]). */
STAGE_API int stage_op_kv4_debug_stall(int calls);

#ifdef __cplusplus
}
#endif
#endif /* LAYER_RANGE_STAGE_KV4_H */
