// Entry points of include/stage_step.h: argument checks and launches of the step's operators.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>

#include "../../include/stage_step.h"
#include "ops_error.h"
#include "step.cuh"

using lrs::op_cuda;
using lrs::op_err;
using lrs::op_host_failure;

static_assert(lrs::kTypeF32 == STAGE_F32 && lrs::kTypeF16 == STAGE_F16 && lrs::kTypeBf16 == STAGE_BF16, "types");

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool known_dtype(int dtype) { return dtype == STAGE_F32 || dtype == STAGE_F16 || dtype == STAGE_BF16; }
int elem_bytes(int dtype) { return dtype == STAGE_F32 ? 4 : 2; }
constexpr int kMaxRows = 1 << 24;
thread_local int g_stall = 0, g_late = 0;  // calls of stage_op_f8_gemm that are to run out of time (tests)

// Rows of `width` elements at a stride; int64 products cannot overflow within these bounds.
int check_rows(const void* p, int64_t stride, int64_t width, int bytes, const char* what) {
  if (!p) return op_err(STAGE_E_INVALID, "null %s", what);
  if (!aligned(p, bytes)) return op_err(STAGE_E_INVALID, "%s must be aligned to its elements", what);
  if (stride < width || stride > ((int64_t)1 << 32))
    return op_err(STAGE_E_INVALID, "the row stride of %s must be from %lld to 2^32 elements", what, (long long)width);
  return STAGE_OK;
}

// Whether rows at this base and stride (elements) begin at multiples of `unit` bytes.
bool rows_at(const void* p, int64_t stride, int bytes, int unit) { return aligned(p, unit) && stride * bytes % unit == 0; }

}  // namespace

extern "C" {

int stage_op_norm_f8(const void* x_dev, int x_dtype, int64_t x_stride, const void* resid_dev, int resid_dtype,
                     int64_t resid_stride, void* resid_out_dev, int64_t resid_out_stride, const float* gamma_dev, float eps,
                     int n_tok, int n, void* q_dev, int64_t q_stride, float* scale_dev, int64_t scale_stride, void* y_dev,
                     int64_t y_stride, void* stream) try {
  if (!known_dtype(x_dtype)) return op_err(STAGE_E_INVALID, "unknown dtype %d", x_dtype);
  if (n_tok < 0 || n_tok > kMaxRows) return op_err(STAGE_E_INVALID, "n_tok outside [0, 2^24]");
  if (n < 1 || n > 32768) return op_err(STAGE_E_INVALID, "n outside [1, 32768]");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return op_err(STAGE_E_INVALID, "eps must be finite and not negative");
  if (!resid_dev != !resid_out_dev) return op_err(STAGE_E_INVALID, "resid and resid_out go together");
  if (resid_dev && resid_dtype != x_dtype && resid_dtype != STAGE_F32)
    return op_err(STAGE_E_INVALID, "resid must have x's type or float32");
  if (!q_dev != !scale_dev) return op_err(STAGE_E_INVALID, "q and scale go together");
  if (!q_dev && !y_dev && n_tok) return op_err(STAGE_E_INVALID, "no output");
  if (n_tok == 0) return STAGE_OK;
  const int xb = elem_bytes(x_dtype), rb = elem_bytes(resid_dtype);
  if (int rc = check_rows(x_dev, x_stride, n, xb, "x")) return rc;
  bool vec = rows_at(x_dev, x_stride, xb, 4 * xb);
  if (resid_dev) {
    if (int rc = check_rows(resid_dev, resid_stride, n, rb, "resid")) return rc;
    if (int rc = check_rows(resid_out_dev, resid_out_stride, n, rb, "resid_out")) return rc;
    if (resid_dev == resid_out_dev && resid_stride != resid_out_stride)
      return op_err(STAGE_E_INVALID, "resid_out in resid's place must have its stride");
    vec = vec && rows_at(resid_dev, resid_stride, rb, 4 * rb) && rows_at(resid_out_dev, resid_out_stride, rb, 4 * rb);
  }
  if (gamma_dev) {
    if (!aligned(gamma_dev, 4)) return op_err(STAGE_E_INVALID, "gamma must be 4-byte aligned");
    vec = vec && aligned(gamma_dev, 16);
  }
  if (q_dev) {
    if (int rc = check_rows(q_dev, q_stride, n, 1, "q")) return rc;
    if (int rc = check_rows(scale_dev, scale_stride, n_tok, 4, "scale")) return rc;
    vec = vec && rows_at(q_dev, q_stride, 1, 4);
  }
  if (y_dev) {
    if (int rc = check_rows(y_dev, y_stride, n, xb, "y")) return rc;
    vec = vec && rows_at(y_dev, y_stride, xb, 4 * xb);
  }
  lrs::NormF8Args a;
  a.x = x_dev;
  a.resid = resid_dev;
  a.resid_out = resid_out_dev;
  a.gamma = gamma_dev;
  a.q = (uint8_t*)q_dev;
  a.scale = scale_dev;
  a.y = y_dev;
  a.x_stride = x_stride;
  a.resid_stride = resid_stride;
  a.resid_out_stride = resid_out_stride;
  a.q_stride = q_stride;
  a.scale_stride = scale_stride;
  a.y_stride = y_stride;
  a.n_tok = n_tok;
  a.n = n;
  a.eps = eps;
  a.vec = vec;
  const cudaError_t e = lrs::launch_norm_f8(a, x_dtype, resid_dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? STAGE_OK : op_cuda(e, "norm f8");
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_f8_gemm(const void* a_dev, int64_t a_stride, const float* a_scale_dev, int64_t a_scale_stride, const void* w_dev,
                     int64_t w_stride, const float* w_scale_dev, int M, int N, int K, void* y_dev, int y_dtype, int64_t y_stride,
                     int32_t* error_dev, void* stream) try {
  if (!known_dtype(y_dtype)) return op_err(STAGE_E_INVALID, "unknown dtype %d", y_dtype);
  if (M < 0 || M > kMaxRows || N < 1 || N > kMaxRows || K < 1 || K > (1 << 20))
    return op_err(STAGE_E_INVALID, "sizes: M in [0, 2^24], N in [1, 2^24], K in [1, 2^20]");
  if ((int64_t)M * N > ((int64_t)1 << 40)) return op_err(STAGE_E_INVALID, "M * N above 2^40");
  if (M == 0) return STAGE_OK;
  if (int rc = check_rows(a_dev, a_stride, K, 1, "a")) return rc;
  if (int rc = check_rows(w_dev, w_stride, K, 1, "w")) return rc;
  if (!rows_at(a_dev, a_stride, 1, 16) || !rows_at(w_dev, w_stride, 1, 16))
    return op_err(STAGE_E_INVALID, "a, w and their row strides must be multiples of 16 bytes");
  if (int rc = check_rows(a_scale_dev, a_scale_stride, M, 4, "a_scale")) return rc;
  if (!w_scale_dev || !aligned(w_scale_dev, 4)) return op_err(STAGE_E_INVALID, "null or unaligned w_scale");
  const int yb = elem_bytes(y_dtype);
  if (int rc = check_rows(y_dev, y_stride, N, yb, "y")) return rc;
  if (!aligned(error_dev, 4)) return op_err(STAGE_E_INVALID, "error must be 4-byte aligned");
  lrs::F8GemmArgs g;
  g.a = (const uint8_t*)a_dev;
  g.w = (const uint8_t*)w_dev;
  g.sa = a_scale_dev;
  g.sw = w_scale_dev;
  g.y = y_dev;
  g.error = error_dev;
  g.a_stride = a_stride;
  g.w_stride = w_stride;
  g.sa_stride = a_scale_stride;
  g.y_stride = y_stride;
  g.M = M;
  g.N = N;
  g.K = K;
  g.nkb = (K + 127) / 128;
  g.vec = rows_at(y_dev, y_stride, yb, 16);
  if (g_stall > 0) {
    --g_stall;
    g.stall = lrs::kStallCopies;
  } else if (g_late > 0) {
    --g_late;
    g.stall = lrs::kStallLate;
  }
  const cudaError_t e = lrs::launch_f8_gemm(g, y_dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? STAGE_OK : op_cuda(e, "f8 gemm");
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_f8_debug_stall(int calls) try {
  if (calls < 0 || calls > 16) return op_err(STAGE_E_INVALID, "calls outside [0, 16]");
  g_stall = calls;
  return STAGE_OK;
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_f8_debug_late(int calls) try {
  if (calls < 0 || calls > 16) return op_err(STAGE_E_INVALID, "calls outside [0, 16]");
  g_late = calls;
  return STAGE_OK;
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_rope_freqs(int rot_dim, double theta, int scaling, double factor, double first_len, double low, double high,
                        double* freqs, float* scale) try {
  constexpr double kTwoPi = 6.283185307179586476925;
  if (!freqs || !scale) return op_err(STAGE_E_INVALID, "null pointer");
  if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2) return op_err(STAGE_E_INVALID, "rot_dim must be even, in [2, 1024]");
  if (!(theta > 1.0) || !std::isfinite(theta)) return op_err(STAGE_E_INVALID, "theta must be above 1");
  if (scaling < STAGE_ROPE_PLAIN || scaling > STAGE_ROPE_PARTS) return op_err(STAGE_E_INVALID, "unknown scaling %d", scaling);
  if (scaling != STAGE_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return op_err(STAGE_E_INVALID, "factor must be 1 or more");
  if (scaling == STAGE_ROPE_BASE && rot_dim == 2) return op_err(STAGE_E_INVALID, "no base scaling of a single pair");
  const bool mixed = scaling == STAGE_ROPE_BANDS || scaling == STAGE_ROPE_PARTS;
  if (mixed && (!(first_len >= 1.0) || !std::isfinite(first_len) || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return op_err(STAGE_E_INVALID, "first_len must be 1 or more, and 0 < low < high");
  *scale = 1.f;
  if (scaling == STAGE_ROPE_BASE) theta *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  double from = 0, to = 0;
  if (scaling == STAGE_ROPE_PARTS) {
    // first_len theta^(-2 i / rot_dim) / (2 pi) waves at pair i
    const double per = rot_dim / (2.0 * std::log(theta));
    from = std::max(0.0, std::floor(per * std::log(first_len / (kTwoPi * high))));
    to = std::min(rot_dim - 1.0, std::ceil(per * std::log(first_len / (kTwoPi * low))));
    *scale = (float)(0.1 * std::log(factor) + 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(theta, -2.0 * i / rot_dim);
    double keep = 1.0;  // the share of f that stays; the rest is divided by the factor
    if (scaling == STAGE_ROPE_LINEAR) keep = 0.0;
    if (scaling == STAGE_ROPE_BANDS) keep = std::min(1.0, std::max(0.0, (first_len * f / kTwoPi - low) / (high - low)));
    if (scaling == STAGE_ROPE_PARTS) keep = 1.0 - std::min(1.0, std::max(0.0, (i - from) / std::max(to - from, 1e-3)));
    freqs[i] = keep == 1.0 ? f : f * (keep + (1.0 - keep) / factor);
  }
  return STAGE_OK;
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_rope(const void* q_dev, int64_t q_stride, int n_q_heads, const void* k_dev, int64_t k_stride, int n_k_heads,
                  int head_dim, int dtype, const int32_t* pos_dev, int n_tok, const double* freqs_dev, int rot_dim,
                  int interleaved, float scale, void* q_out_dev, int64_t q_out_stride, void* k_out_dev, int64_t k_out_stride,
                  void* stream) try {
  if (!known_dtype(dtype)) return op_err(STAGE_E_INVALID, "unknown dtype %d", dtype);
  if (n_tok < 0 || n_tok > kMaxRows) return op_err(STAGE_E_INVALID, "n_tok outside [0, 2^24]");
  if (n_q_heads < 1 || n_q_heads > 1024 || n_k_heads < 0 || n_k_heads > 1024)
    return op_err(STAGE_E_INVALID, "n_q_heads outside [1, 1024] or n_k_heads outside [0, 1024]");
  if (head_dim < 2 || head_dim > 1024 || rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
    return op_err(STAGE_E_INVALID, "head_dim outside [2, 1024], or rot_dim odd or outside [2, head_dim]");
  if (!std::isfinite(scale)) return op_err(STAGE_E_INVALID, "scale must be finite");
  if (n_tok == 0) return STAGE_OK;
  const int eb = elem_bytes(dtype);
  if (int rc = check_rows(q_dev, q_stride, (int64_t)n_q_heads * head_dim, eb, "q")) return rc;
  if (int rc = check_rows(q_out_dev, q_out_stride, (int64_t)n_q_heads * head_dim, eb, "q_out")) return rc;
  if (q_dev == q_out_dev && q_stride != q_out_stride) return op_err(STAGE_E_INVALID, "q_out in q's place must have its stride");
  bool copy = q_dev != q_out_dev;
  if (n_k_heads) {
    if (int rc = check_rows(k_dev, k_stride, (int64_t)n_k_heads * head_dim, eb, "k")) return rc;
    if (int rc = check_rows(k_out_dev, k_out_stride, (int64_t)n_k_heads * head_dim, eb, "k_out")) return rc;
    if (k_dev == k_out_dev && k_stride != k_out_stride) return op_err(STAGE_E_INVALID, "k_out in k's place must have its stride");
    copy = copy || k_dev != k_out_dev;
  }
  if (!pos_dev || !aligned(pos_dev, 4)) return op_err(STAGE_E_INVALID, "null or unaligned pos");
  if (!freqs_dev || !aligned(freqs_dev, 8)) return op_err(STAGE_E_INVALID, "null or unaligned freqs");
  // whether everything allows accesses of `width` elements
  auto by = [&](int width) {
    const int unit = width * eb;
    return rows_at(q_dev, q_stride, eb, unit) && rows_at(q_out_dev, q_out_stride, eb, unit) &&
           (!n_k_heads || (rows_at(k_dev, k_stride, eb, unit) && rows_at(k_out_dev, k_out_stride, eb, unit))) && head_dim % width == 0 &&
           rot_dim % (interleaved ? width : 2 * width) == 0;
  };
  lrs::RopeArgs a;
  a.q = q_dev;
  a.k = k_dev;
  a.q_out = q_out_dev;
  a.k_out = k_out_dev;
  a.pos = pos_dev;
  a.freqs = freqs_dev;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.hq = n_q_heads;
  a.hk = n_k_heads;
  a.head_dim = head_dim;
  a.rot = rot_dim;
  a.n_tok = n_tok;
  a.interleaved = interleaved != 0;
  a.scale = scale;
  a.vec = by(16 / eb) ? 2 : by(2) ? 1 : 0;
  a.copy = copy && rot_dim < head_dim;
  const cudaError_t e = lrs::launch_rope(a, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? STAGE_OK : op_cuda(e, "rope");
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

int stage_op_logprobs(const void* logits_dev, int dtype, int64_t row_stride, int n_rows, int vocab, const int32_t* tokens_dev,
                      float* logprob_dev, float* entropy_dev, int32_t* rank_dev, int n_top, int32_t* top_ids_dev,
                      float* top_logprobs_dev, void* stream) try {
  if (!known_dtype(dtype)) return op_err(STAGE_E_INVALID, "unknown dtype %d", dtype);
  if (n_rows < 0 || n_rows > kMaxRows) return op_err(STAGE_E_INVALID, "n_rows outside [0, 2^24]");
  if (vocab < 1 || vocab > (1 << 19)) return op_err(STAGE_E_INVALID, "vocab outside [1, 2^19]");
  if (n_top < 0 || n_top > STAGE_LOGPROBS_MAX_TOP || n_top > vocab)
    return op_err(STAGE_E_INVALID, "n_top must be at most %d, and vocab", STAGE_LOGPROBS_MAX_TOP);
  if (!tokens_dev && (logprob_dev || rank_dev)) return op_err(STAGE_E_INVALID, "logprob and rank need tokens");
  if (n_rows == 0) return STAGE_OK;
  if (int rc = check_rows(logits_dev, row_stride, vocab, elem_bytes(dtype), "logits")) return rc;
  const void* all[] = {tokens_dev, logprob_dev, entropy_dev, rank_dev, top_ids_dev, top_logprobs_dev};
  for (const void* p : all)
    if (!aligned(p, 4)) return op_err(STAGE_E_INVALID, "tokens and outputs must be 4-byte aligned");
  lrs::LogprobsArgs a;
  a.z = logits_dev;
  a.tokens = tokens_dev;
  a.logprob = logprob_dev;
  a.entropy = entropy_dev;
  a.rank = rank_dev;
  a.top_ids = top_ids_dev;
  a.top_lp = top_logprobs_dev;
  a.stride = row_stride;
  a.rows = n_rows;
  a.vocab = vocab;
  a.top = top_ids_dev || top_logprobs_dev ? n_top : 0;
  const cudaError_t e = lrs::launch_logprobs(a, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? STAGE_OK : op_cuda(e, "logprobs");
} catch (const std::exception& ex) {
  return op_host_failure(ex.what());
} catch (...) {
  return op_host_failure("unknown exception");
}

}  // extern "C"
