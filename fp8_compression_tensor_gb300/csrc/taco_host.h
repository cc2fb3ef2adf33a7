// taco_host.h -- host-side helpers shared by the C ABI's source files
// (internal to the library): per-device set-up, errors and pointer checks.
#pragma once

#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "taco.h"

namespace taco {

struct DeviceState {
    std::once_flag once;
    cudaError_t init_error = cudaSuccess;
    int sm_count = 0;
    uint32_t *fault = nullptr;  // device address of the fault flags
    int ctas_per_sm = 0;        // last occupancy query (set-up check only)
    std::once_flag train_once;  // set-up of the training operators' kernels
    cudaError_t train_error = cudaSuccess;
    std::once_flag rms_once, gated_once;
    cudaError_t rms_error = cudaSuccess, gated_error = cudaSuccess;
};

// Set-up of the current device, once per device and process.
taco_status_t device_state(DeviceState **out);

// Notes the error for taco_last_cuda_error() and returns TACO_ERR_CUDA.
taco_status_t cuda_fail(cudaError_t e);

bool block_supported(int block);

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime.
cudaError_t tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000 *out);

inline bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

inline bool overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

}  // namespace taco
