// Entry points of include/stage_kv4.h: argument checks and launches of the paged 4-bit cache's kernels.
#include <cuda_runtime.h>

#include <cmath>
#include <exception>

#include "../../include/stage_kv4.h"
#include "kv4.cuh"
#include "ops_error.h"

using lrs::op_cuda;
using lrs::op_err;
using lrs::op_host_failure;

static_assert(lrs::kKv4ErrorAt == STAGE_KV4_ERROR_AT, "stage_kv4.h says where the error word lies");

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool cache_sizes_ok(int64_t n_pages, int page_len, int n_kv_heads, int head_dim) {
  return n_pages >= 1 && page_len >= 16 && page_len <= 4096 && page_len % 16 == 0 && n_pages <= INT32_MAX / page_len &&
         n_kv_heads >= 1 && n_kv_heads <= 1024 && (head_dim == 64 || head_dim == 128);
}

bool known_dtype(int dtype) { return dtype == STAGE_F32 || dtype == STAGE_F16 || dtype == STAGE_BF16; }

bool attention_sizes_ok(int n_seqs, int n_q_heads, int n_kv_heads, int head_dim, int max_q, int max_len) {
  return n_seqs >= 0 && n_seqs <= 65535 && n_kv_heads >= 1 && n_q_heads >= 1 && n_q_heads <= 1024 && n_q_heads % n_kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128) && max_q >= 1 && max_q <= (1 << 20) && max_len >= 1 && max_len <= (1 << 30);
}

// A sequence has no more tokens than the call.
int bounded_q(int max_q, int n_tok) { return max_q < n_tok ? max_q : n_tok; }

int check_cache(const void* cache, int64_t n_pages, int page_len, int n_kv_heads, int head_dim, int dtype, int n_tok) {
  if (!cache_sizes_ok(n_pages, page_len, n_kv_heads, head_dim))
    return op_err(STAGE_E_INVALID,
                  "cache sizes: n_pages >= 1, page_len a multiple of 16 up to 4096, n_pages * page_len < 2^31, "
                  "1 to 1024 KV heads, head_dim 64 or 128");
  if (!known_dtype(dtype)) return op_err(STAGE_E_INVALID, "unknown dtype %d", dtype);
  if (n_tok < 0 || n_tok > (1 << 24)) return op_err(STAGE_E_INVALID, "n_tok outside [0, 2^24]");
  if (!cache) return op_err(STAGE_E_INVALID, "null cache");
  if (!aligned(cache, 16)) return op_err(STAGE_E_INVALID, "the cache must be 16-byte aligned");
  return STAGE_OK;
}

int elem_bytes(int dtype) { return dtype == STAGE_F32 ? 4 : 2; }

// Rows of `width` elements at a stride; int64 products cannot overflow within these bounds.
int check_rows(const void* p, int64_t stride, int64_t width, int dtype, const char* what) {
  if (!p) return op_err(STAGE_E_INVALID, "null %s", what);
  if (!aligned(p, 16)) return op_err(STAGE_E_INVALID, "%s must be 16-byte aligned", what);
  if (stride < width || stride > ((int64_t)1 << 32) || stride * elem_bytes(dtype) % 16)
    return op_err(STAGE_E_INVALID, "the row stride of %s must be a multiple of 16 bytes, from %lld to 2^32 elements", what,
                  (long long)width);
  return STAGE_OK;
}

lrs::Kv4Cache make_cache(const void* data, int64_t n_pages, int page_len, int n_kv_heads) {
  lrs::Kv4Cache c;
  c.data = (uint8_t*)data;
  c.n_pages = n_pages;
  c.page_len = page_len;
  c.n_kv_heads = n_kv_heads;
  return c;
}

}  // namespace

extern "C" {

size_t stage_op_kv4_cache_bytes(int64_t n_pages, int page_len, int n_kv_heads, int head_dim) {
  if (!cache_sizes_ok(n_pages, page_len, n_kv_heads, head_dim)) return 0;
  return (size_t)n_pages * n_kv_heads * (page_len / 16) * lrs::kv4_tile_bytes(head_dim);
}

int stage_op_kv4_plan(int n_seqs, int page_len, int64_t n_pages, const int32_t* seq_len_dev, const int32_t* keep_len_dev,
                      const int32_t* new_len_dev, int32_t* table_dev, int table_stride, int32_t* free_ring_dev, int ring_len,
                      const int32_t* free_state_dev, int32_t* seq_len_out_dev, int32_t* free_state_out_dev, int n_tok,
                      int32_t* cu_new_dev, int32_t* slot_dev, int32_t* pos_dev, int32_t* seq_dev, int32_t* status_dev,
                      void* stream) try {
  if (n_seqs < 0 || n_seqs > 65536) return op_err(STAGE_E_INVALID, "n_seqs outside [0, 65536]");
  if (page_len < 16 || page_len > 4096 || page_len % 16)
    return op_err(STAGE_E_INVALID, "page_len must be a multiple of 16 up to 4096");
  if (n_pages < 1 || n_pages > INT32_MAX / page_len) return op_err(STAGE_E_INVALID, "n_pages * page_len outside [1, 2^31)");
  if (table_stride < 1 || table_stride > (1 << 20)) return op_err(STAGE_E_INVALID, "table_stride outside [1, 2^20]");
  if (ring_len < 1 || ring_len > (1 << 30)) return op_err(STAGE_E_INVALID, "ring_len outside [1, 2^30]");
  if (n_tok < 0 || n_tok > (1 << 24)) return op_err(STAGE_E_INVALID, "n_tok outside [0, 2^24]");
  if (!free_ring_dev || !free_state_dev || !free_state_out_dev || !cu_new_dev || !status_dev ||
      (n_seqs && (!seq_len_dev || !new_len_dev || !table_dev || !seq_len_out_dev)) ||
      (n_tok && (!slot_dev || !pos_dev || !seq_dev)))
    return op_err(STAGE_E_INVALID, "null pointer");
  const void* all[] = {seq_len_dev, keep_len_dev, new_len_dev, table_dev, free_ring_dev, free_state_dev, seq_len_out_dev,
                       free_state_out_dev, cu_new_dev, slot_dev, pos_dev, seq_dev, status_dev};
  for (const void* p : all)
    if (!aligned(p, 4)) return op_err(STAGE_E_INVALID, "int32 arrays must be 4-byte aligned");
  lrs::Kv4PlanArgs a;
  a.n_seqs = n_seqs;
  a.page_len = page_len;
  a.n_pages = n_pages;
  a.table_stride = table_stride;
  a.ring_len = ring_len;
  a.n_tok = n_tok;
  a.seq_len = seq_len_dev;
  a.keep_len = keep_len_dev;
  a.new_len = new_len_dev;
  a.table = table_dev;
  a.ring = free_ring_dev;
  a.free_state = free_state_dev;
  a.seq_len_out = seq_len_out_dev;
  a.free_state_out = free_state_out_dev;
  a.cu_new = cu_new_dev;
  a.slot = slot_dev;
  a.pos = pos_dev;
  a.seq = seq_dev;
  a.status = status_dev;
  const cudaError_t e = lrs::launch_kv4_plan(a, (cudaStream_t)stream);
  return e == cudaSuccess ? STAGE_OK : op_cuda(e, "kv4 plan");
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_kv4_append(void* cache_dev, int64_t n_pages, int page_len, int n_kv_heads, int head_dim, const void* k_dev,
                        const void* v_dev, int dtype, int64_t row_stride, const int32_t* slot_dev, int n_tok,
                        void* stream) try {
  if (int rc = check_cache(cache_dev, n_pages, page_len, n_kv_heads, head_dim, dtype, n_tok)) return rc;
  if (n_tok == 0) return STAGE_OK;
  if (int rc = check_rows(k_dev, row_stride, (int64_t)n_kv_heads * head_dim, dtype, "k")) return rc;
  if (int rc = check_rows(v_dev, row_stride, (int64_t)n_kv_heads * head_dim, dtype, "v")) return rc;
  if (!slot_dev || !aligned(slot_dev, 4)) return op_err(STAGE_E_INVALID, "null or unaligned slot");
  lrs::Kv4RowsArgs a;
  a.c = make_cache(cache_dev, n_pages, page_len, n_kv_heads);
  a.k_in = k_dev;
  a.v_in = v_dev;
  a.row_stride = row_stride;
  a.slot = slot_dev;
  a.n_tok = n_tok;
  const cudaError_t e = lrs::launch_kv4_append(a, head_dim, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? STAGE_OK : op_cuda(e, "kv4 append");
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_kv4_read(const void* cache_dev, int64_t n_pages, int page_len, int n_kv_heads, int head_dim,
                      const int32_t* slot_dev, int n_tok, void* k_out_dev, void* v_out_dev, int dtype, int64_t row_stride,
                      void* stream) try {
  if (int rc = check_cache(cache_dev, n_pages, page_len, n_kv_heads, head_dim, dtype, n_tok)) return rc;
  if (n_tok == 0) return STAGE_OK;
  if (int rc = check_rows(k_out_dev, row_stride, (int64_t)n_kv_heads * head_dim, dtype, "k_out")) return rc;
  if (int rc = check_rows(v_out_dev, row_stride, (int64_t)n_kv_heads * head_dim, dtype, "v_out")) return rc;
  if (!slot_dev || !aligned(slot_dev, 4)) return op_err(STAGE_E_INVALID, "null or unaligned slot");
  lrs::Kv4RowsArgs a;
  a.c = make_cache(cache_dev, n_pages, page_len, n_kv_heads);
  a.k_out = k_out_dev;
  a.v_out = v_out_dev;
  a.row_stride = row_stride;
  a.slot = slot_dev;
  a.n_tok = n_tok;
  const cudaError_t e = lrs::launch_kv4_read(a, head_dim, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? STAGE_OK : op_cuda(e, "kv4 read");
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_kv4_attention_many(int n_seqs, int n_tok, int n_q_heads, int n_kv_heads, int head_dim, int dtype, int max_q,
                                int max_len) try {
  if (!attention_sizes_ok(n_seqs, n_q_heads, n_kv_heads, head_dim, max_q, max_len) || n_kv_heads > 1024 || !known_dtype(dtype) ||
      n_tok < 0 || n_tok > (1 << 24))
    return op_err(STAGE_E_INVALID, "no attention of these sizes");
  lrs::Kv4AttnArgs a;
  a.c.n_kv_heads = n_kv_heads;
  a.n_q_heads = n_q_heads;
  a.n_seqs = n_seqs;
  a.max_q = bounded_q(max_q, n_tok);
  a.max_len = max_len;
  return n_tok && n_seqs && lrs::kv4_many_columns(a, head_dim, dtype);
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

size_t stage_op_kv4_attention_workspace_bytes(int n_seqs, int n_q_heads, int n_kv_heads, int head_dim, int max_q,
                                              int max_len) {
  if (!attention_sizes_ok(n_seqs, n_q_heads, n_kv_heads, head_dim, max_q, max_len)) return 0;
  return lrs::kv4_attention_ws_bytes(n_seqs, n_q_heads, n_kv_heads, head_dim, max_q, max_len);
}

int stage_op_kv4_attention(const void* cache_dev, int64_t n_pages, int page_len, int n_kv_heads, int head_dim,
                           const void* q_dev, int dtype, int64_t q_stride, int n_tok, int n_q_heads,
                           const int32_t* cu_q_dev, const int32_t* seq_len_dev, const int32_t* table_dev, int table_stride,
                           int n_seqs, int max_q, int max_len, void* out_dev, int64_t out_stride, void* workspace_dev,
                           size_t workspace_bytes, void* stream) try {
  if (int rc = check_cache(cache_dev, n_pages, page_len, n_kv_heads, head_dim, dtype, n_tok)) return rc;
  if (n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % n_kv_heads)
    return op_err(STAGE_E_INVALID, "n_q_heads must be a multiple of n_kv_heads, at most 1024");
  if (n_seqs < 0 || n_seqs > 65535) return op_err(STAGE_E_INVALID, "n_seqs outside [0, 65535]");
  if (max_q < 1 || max_q > (1 << 20) || max_len < 1 || max_len > (1 << 30))
    return op_err(STAGE_E_INVALID, "max_q outside [1, 2^20] or max_len outside [1, 2^30]");
  if (table_stride < 1 || table_stride > (1 << 20)) return op_err(STAGE_E_INVALID, "table_stride outside [1, 2^20]");
  if (n_tok == 0 || n_seqs == 0) return STAGE_OK;
  if (int rc = check_rows(q_dev, q_stride, (int64_t)n_q_heads * head_dim, dtype, "q")) return rc;
  if (int rc = check_rows(out_dev, out_stride, (int64_t)n_q_heads * head_dim, dtype, "out")) return rc;
  if (!cu_q_dev || !seq_len_dev || !table_dev || !aligned(cu_q_dev, 4) || !aligned(seq_len_dev, 4) || !aligned(table_dev, 4))
    return op_err(STAGE_E_INVALID, "null or unaligned cu_q, seq_len or table");
  const size_t need = stage_op_kv4_attention_workspace_bytes(n_seqs, n_q_heads, n_kv_heads, head_dim, max_q, max_len);
  if (!workspace_dev || workspace_bytes < need || !aligned(workspace_dev, 16))
    return op_err(STAGE_E_INVALID, "workspace must be 16-byte aligned and hold %zu bytes", need);
  lrs::Kv4AttnArgs a;
  a.c = make_cache(cache_dev, n_pages, page_len, n_kv_heads);
  a.q = q_dev;
  a.out = out_dev;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.n_tok = n_tok;
  a.n_q_heads = n_q_heads;
  a.n_seqs = n_seqs;
  a.table_stride = table_stride;
  a.max_q = bounded_q(max_q, n_tok);
  a.max_len = max_len;
  a.cu_q = cu_q_dev;
  a.seq_len = seq_len_dev;
  a.table = table_dev;
  a.scale = (float)(1.0 / std::sqrt((double)head_dim));
  a.ws = workspace_dev;
  const cudaError_t e = lrs::launch_kv4_attention(a, head_dim, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? STAGE_OK : op_cuda(e, "kv4 attention");
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_kv4_debug_stall(int calls) try {
  if (calls < 0 || calls > 16) return op_err(STAGE_E_INVALID, "calls outside [0, 16]");
  lrs::kv4_stall(calls);
  return STAGE_OK;
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

}  // extern "C"
