// taco_weight_grad.cu -- weight gradient of a linear layer whose input was
// kept as an 8-bit checkpoint, for GB300 (sm_103a).
//
//   dW[m, n] = scale[n] sum_r dY[r, m] X[r, n] + dy_sum[m] shift[n]  [+ dW before]
//
// with X the values of the records and dY the bf16 gradient of the layer's
// output.  scale and shift (a layer norm's weight and bias) turn the records
// of the normalised input xhat into those of the norm's output xhat scale +
// shift without decoding them twice: both act per column n, so they leave the
// sum over rows and join the epilogue; dy_sum[m] = sum_r dY[r, m] is the
// layer's bias gradient.
#include <climits>

#include "taco_kernels.h"
#include "taco_train.cuh"

namespace taco {
namespace {

constexpr int kTile = 64, kDepth = 16;

__device__ __forceinline__ void finish_element(const WeightGradArgs &a, int64_t m, int64_t n, float v)
{
    if (a.scale)
        v *= load_param(a.scale, a.param_dtype, n);
    if (a.shift)
        v = fmaf(a.dy_sum[m], load_param(a.shift, a.param_dtype, n), v);
    const int64_t i = m * a.hidden + n;
    if (a.accumulate)
        v += load_param(a.dw, a.dtype, i);
    store_param(a.dw, a.dtype, i, v);
}

// 64 x 64 tiles of dW on the CUDA cores, 4 x 4 values a thread, any out width.
__global__ void __launch_bounds__(256) taco_weight_grad_any_kernel(WeightGradArgs a)
{
    __shared__ float sa[kDepth][kTile], sb[kDepth][kTile];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t across = (a.hidden + kTile - 1) / kTile;
    const int64_t m0 = blockIdx.x / across * kTile, n0 = blockIdx.x % across * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const __nv_bfloat16 *dy = static_cast<const __nv_bfloat16 *>(a.dy);
    float acc[4][4] = {};
    for (int64_t r0 = 0; r0 < a.rows; r0 += kDepth) {
        __syncthreads();
        for (int i = threadIdx.x; i < kDepth * kTile; i += 256) {
            const int64_t r = r0 + i / kTile, m = m0 + i % kTile, n = n0 + i % kTile;
            sa[i / kTile][i % kTile] = r < a.rows && m < a.out ? __bfloat162float(dy[r * a.out + m]) : 0.f;
            sb[i / kTile][i % kTile] =
                r < a.rows && n < a.hidden ? record_value(a.packed, r * a.hidden + n, a.block, a.code) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; k++) {
            float x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[j] = sa[k][ty * 4 + j];
                y[j] = sb[k][tx * 4 + j];
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
        }
    }
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++)
            if (m0 + ty * 4 + i < a.out && n0 + tx * 4 + j < a.hidden)
                finish_element(a, m0 + ty * 4 + i, n0 + tx * 4 + j, acc[i][j]);
}

}  // namespace

int weight_grad_splits(int64_t, int64_t, int64_t) { return 1; }

bool weight_grad_in_range(int64_t rows, int64_t out, int64_t hidden)
{
    return rows <= INT32_MAX && (out + kTile - 1) / kTile <= INT32_MAX / ((hidden + kTile - 1) / kTile + 1);
}

cudaError_t launch_weight_grad(const WeightGradArgs &a, uint32_t *, int, cudaStream_t stream)
{
    WeightGradArgs args = a;
    void *p[] = {&args};
    const int64_t tiles = (a.hidden + kTile - 1) / kTile * ((a.out + kTile - 1) / kTile);
    return launch_kernel(reinterpret_cast<void *>(&taco_weight_grad_any_kernel), static_cast<int>(tiles), 256, 0, stream, p);
}

}  // namespace taco
