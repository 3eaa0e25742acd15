// The paged 4-bit KV cache: its layout and the launch interface of its kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lrs {

// [page][kv head][tile of 16 positions][tile bytes]; a tile is K codes, K scales, V codes, V scales
// (include/stage_kv4.h states the order of the codes).
constexpr int kKv4Tile = 16;
__host__ __device__ constexpr int kv4_codes(int D) { return kKv4Tile * D / 2; }        // bytes of a tile's K (or V) codes
__host__ __device__ constexpr int kv4_scales(int D) { return kKv4Tile * (D / 32) * 2; }  // bytes of its scales
__host__ __device__ constexpr int kv4_half(int D) { return kv4_codes(D) + kv4_scales(D); }
__host__ __device__ constexpr int kv4_tile_bytes(int D) { return 2 * kv4_half(D); }

// Byte offsets inside a tile's K (V) codes of the two bytes that hold the four dims 32 * block + 4 * l .. + 3
// of position p.
template <int D>
__device__ __forceinline__ int kv4_k_off(int p, int block, int l) {
  return p * (D / 2) + (l >> 1) * (D / 8) + block * 4 + (l & 1) * 2;
}
template <int D>
__device__ __forceinline__ int kv4_v_off(int p, int block, int l) {
  return (((p >> 3) * 8 + l) * 4 + ((p >> 1) & 3)) * (D / 8) + (p & 1) * (D / 16) + block * 2;
}

struct Kv4Cache {
  uint8_t* data = nullptr;
  long long n_pages = 0;
  int page_len = 0, n_kv_heads = 0;
};

enum Kv4Type { KV4_F32 = 0, KV4_F16 = 1, KV4_BF16 = 2 };

struct Kv4PlanArgs {
  int n_seqs = 0, page_len = 0, table_stride = 0, ring_len = 0, n_tok = 0;
  long long n_pages = 0;
  const int* seq_len = nullptr;
  const int* keep_len = nullptr;  // may be null
  const int* new_len = nullptr;
  int* table = nullptr;
  int* ring = nullptr;
  const int* free_state = nullptr;
  int* seq_len_out = nullptr;
  int* free_state_out = nullptr;
  int* cu_new = nullptr;
  int* slot = nullptr;
  int* pos = nullptr;
  int* seq = nullptr;
  int* status = nullptr;
};
cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, cudaStream_t st);

struct Kv4RowsArgs {
  Kv4Cache c;
  const void* k_in = nullptr;  // append
  const void* v_in = nullptr;
  void* k_out = nullptr;       // read
  void* v_out = nullptr;
  long long row_stride = 0;    // elements
  const int* slot = nullptr;
  int n_tok = 0;
};
cudaError_t launch_kv4_append(const Kv4RowsArgs& a, int head_dim, int dtype, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4RowsArgs& a, int head_dim, int dtype, cudaStream_t st);

struct Kv4AttnArgs {
  Kv4Cache c;
  const void* q = nullptr;
  void* out = nullptr;
  long long q_stride = 0, out_stride = 0;
  int n_tok = 0, n_q_heads = 0, n_seqs = 0, table_stride = 0, max_q = 0, max_len = 0;
  const int* cu_q = nullptr;
  const int* seq_len = nullptr;
  const int* table = nullptr;
  float scale = 1.f;
  void* ws = nullptr;
};
cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int head_dim, int dtype, cudaStream_t st);
// Workspace: arrival counters, zero between calls, which calls of many columns leave alone; the error word, in a
// line of its own; then partial results.
constexpr int kKv4MaxCtas = 512;
constexpr size_t kKv4ErrorAt = kKv4MaxCtas * sizeof(unsigned), kKv4CounterBytes = kKv4ErrorAt + 128;
__device__ __forceinline__ int* kv4_error_word(void* ws) { return reinterpret_cast<int*>((char*)ws + kKv4ErrorAt); }
// Row tiles times parts that the workspace of a chunk call holds.
constexpr int kKv4ChunkParts = 192;
size_t kv4_chunk_ws_bytes(int head_dim);
void kv4_stall(int calls);  // the thread's next calls of many columns copy nothing of the cache
cudaError_t launch_kv4_chunk(const Kv4AttnArgs& a, int head_dim, int dtype, cudaStream_t st);
// Row tiles at a call's bounds times KV heads times sequences, at most, for the kernel for many columns, whose CTAs look through them.
constexpr long long kKv4ChunkItems = 1ll << 30;
// Whether a call runs on the kernel for many columns.
bool kv4_many_columns(const Kv4AttnArgs& a, int head_dim, int dtype);
size_t kv4_attention_ws_bytes(int n_seqs, int n_q_heads, int n_kv_heads, int head_dim, int max_q, int max_len);

}  // namespace lrs
