// status.h -- a CUDA call's result as the library's status.
#pragma once

#include <cuda_runtime.h>

#include "moe_qmm.h"

namespace moe {

// A refused launch stays the thread's last error, and the launch checks of the next call would
// take it for their own: it is taken away here.
inline moe_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
}

}  // namespace moe
