// taco_train.h -- host-side view of the training operators' kernels (internal
// to the library).  Every launch function expects validated arguments.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "taco_kernels.h"

namespace taco {

// Element types (taco_dtype_t).
constexpr int kTypeBf16 = 0;
constexpr int kTypeF16 = 1;
constexpr int kTypeF32 = 2;

// launch_kernel (taco_kernels.h) with a two-dimensional grid.
inline cudaError_t launch_kernel_2d(const void *fn, unsigned grid_x, unsigned grid_y, int threads, size_t smem,
                                    cudaStream_t stream, void **args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid_x, grid_y);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = TACO_PDL ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Most row chunks whose column sums a backward pass keeps apart (two CTAs on each of 152 SMs).
constexpr int kMaxColumnParts = 304;

struct NormArgs {
    const void *x, *residual, *weight, *bias;   // residual, weight, bias may be null
    void *y, *summed;                           // summed non-null exactly with residual
    float *mean, *rstd;
    uint8_t *packed;                            // null: no records
    int64_t rows, hidden;
    float eps;
    int param_dtype, block, code;
};

struct NormGradArgs {
    const void *dy, *x, *weight, *dsummed;      // x null: from records
    const float *mean, *rstd;
    const uint8_t *packed;
    void *dx;
    float *parts;                               // [2][parts][hidden] column sums of dy * xhat and dy; null: none wanted
    int64_t rows, hidden;
    int param_dtype, block, code, nparts;
};

struct GeluArgs {
    const void *x, *bias;
    void *y;
    uint8_t *packed;
    int64_t rows, hidden;
    int param_dtype, tanh_form, block, code;
};

struct GeluGradArgs {
    const void *dy;
    const uint8_t *packed;
    void *dx, *y;                               // y may be null
    float *parts;                               // [parts][hidden] column sums of dx; null: none wanted
    int64_t rows, hidden;
    int tanh_form, block, code, nparts;
};

struct WeightGradArgs {
    const void *dy;
    const uint8_t *packed;
    void *dw;
    const void *scale, *shift;                  // [hidden] of param_dtype, or null
    const float *dy_sum;                        // [out]
    float *parts;                               // weight_grad_workspace() bytes
    int64_t rows, out, hidden;
    int dtype, param_dtype, accumulate, block, code;
};

// Kernel attributes, once per device.
cudaError_t init_weight_grad();
cudaError_t init_norm();
cudaError_t init_norm_grad();

cudaError_t launch_norm(int dtype, const NormArgs &a, int sms, cudaStream_t stream);
// The gradient launches set nparts to the number of row chunks they use (at most what the caller gives).
cudaError_t launch_norm_grad(int dtype, NormGradArgs *a, int sms, cudaStream_t stream);
cudaError_t launch_gelu(int dtype, const GeluArgs &a, int sms, cudaStream_t stream);
cudaError_t launch_gelu_grad(int dtype, GeluGradArgs *a, int sms, cudaStream_t stream);

// Workspace of a weight gradient and the range its kernels address.
int64_t weight_grad_workspace(int64_t rows, int64_t out, int64_t hidden);
bool weight_grad_in_range(int64_t rows, int64_t out, int64_t hidden);
cudaError_t launch_weight_grad(const WeightGradArgs &a, uint32_t *fault, int sms, cudaStream_t stream);

// out[c] = sum over p < nparts of parts[p][c] in a fixed order; zeros for nparts = 0.  parts holds two
// such arrays ([2][nparts][n]) where out2 takes the second one's sums; either output may be null.
cudaError_t launch_column_sums(const float *parts, int nparts, int64_t n, void *out, void *out2, int dtype,
                               cudaStream_t stream);

}  // namespace taco
