// call.h -- what every C entry point does around its launch (gemm_api.cu).
#pragma once

#include <cuda_runtime.h>

#include "gemm.h"

namespace gemm {

// The name gemm_last_kernel() reports for the calling thread.
void set_last_kernel(const char *name);
// GEMM_OK when the current device runs this library's code.
gemm_status_t check_device_status();
// A launch's CUDA error as a status; records the kernel's name on success.
gemm_status_t finish_call(cudaError_t e, const char *name);

}  // namespace gemm
