// Errors of CUDA calls, shared by the files of the C ABI.
#pragma once

#include <cuda_runtime.h>

namespace hyb {

// Keeps a failed CUDA call's error for hyb_attn_last_cuda_error; returns HYB_ECUDA.
int record_cuda_error(cudaError_t e);

}  // namespace hyb
