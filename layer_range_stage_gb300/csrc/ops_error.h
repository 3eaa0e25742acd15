// The last-error string of the stage_op_* entry points (one per calling thread).
#pragma once

#include <cuda_runtime.h>

namespace lrs {

int op_err(int code, const char* fmt, ...);
int op_cuda(cudaError_t e, const char* where);
// STAGE_E_HOST for a C++ exception that reached an entry point.
int op_host_failure(const char* what) noexcept;

}  // namespace lrs
