// taco_gated.cu -- gated linear layer (both projections, the activation, the
// product and the 8-bit checkpoint of the projections) and its input's gradient,
// for GB300 (sm_103a).
//
//   z = x W^T + bias,  y = act(z_gate) z_up,  dx = dz W
#include <algorithm>
#include <climits>

#include "taco_activation.cuh"
#include "taco_kernels.h"

namespace taco {
namespace {

// out[M, N] = A[M, K] B, B stored as [N, K] or (BT) as [K, N]: tiles of 64 x 64, 4 x 4 a thread, sums in binary32.
template <typename T, typename O, bool BT>
__global__ void __launch_bounds__(256) taco_gated_product_kernel(const T *a, const T *b, O *out, int64_t M, int64_t N, int64_t K)
{
    __shared__ float sa[16][65], sb[16][65];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t tiles_n = (N + 63) / 64, tiles = tiles_n * ((M + 63) / 64);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t m0 = t / tiles_n * 64, n0 = t % tiles_n * 64;
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < K; k0 += 16) {
            for (int i = threadIdx.x; i < 1024; i += 256) {
                const int64_t m = m0 + i / 16, k = k0 + i % 16;
                sa[i % 16][i / 16] = m < M && k < K ? to_float(a[m * K + k]) : 0.f;
                const int64_t n = n0 + (BT ? i % 64 : i / 16), kb = k0 + (BT ? i / 64 : i % 16);
                sb[BT ? i / 64 : i % 16][BT ? i % 64 : i / 16] = n < N && kb < K ? to_float(b[BT ? kb * N + n : n * K + kb]) : 0.f;
            }
            __syncthreads();
            for (int k = 0; k < 16; k++)
                for (int i = 0; i < 4; i++)
                    for (int j = 0; j < 4; j++)
                        acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; i++)
            for (int j = 0; j < 4; j++)
                if (m0 + ty + 16 * i < M && n0 + tx + 16 * j < N)
                    out[(m0 + ty + 16 * i) * N + n0 + tx + 16 * j] = from_float<O>(acc[i][j]);
    }
}

// y and the records of z from z as binary32: a warp takes 256 columns of a row.
template <typename T, int ACT>
__global__ void __launch_bounds__(256) taco_gated_finish_kernel(GatedArgs a, const float *z)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t pieces = (a.inner + 255) / 256, n = a.rows * pieces;
    for (int64_t w = blockIdx.x * 8ll + (threadIdx.x >> 5); w < n; w += gridDim.x * 8ll) {
        const int64_t row = w / pieces, c0 = w % pieces * 256;
        F8 g[1], u[1];
        auto value = [&](int k, int64_t c) {
            if (c >= a.inner)
                return 0.f;
            const float v = z[(row * 2 + k) * a.inner + c];
            return a.bias ? v + load_param(a.bias, a.param_dtype, k * a.inner + c) : v;
        };
        for (int i = 0; i < 4; i++) {
            const int64_t c = c0 + lane * 8 + 2 * i;
            g[0].v[i] = make_float2(value(0, c), value(0, c + 1));
            u[0].v[i] = make_float2(value(1, c), value(1, c + 1));
            const float2 y = mul2(activation2<ACT>(g[0].v[i]), u[0].v[i]);
            if (c < a.inner)
                static_cast<T *>(a.y)[row * a.inner + c] = from_float<T>(y.x);
            if (c + 1 < a.inner)
                static_cast<T *>(a.y)[row * a.inner + c + 1] = from_float<T>(y.y);
        }
        if (a.packed) {
            const int col[1] = {lane * 8}, left = static_cast<int>(a.inner - c0);
            for (int k = 0; k < 2; k++) {
                uint8_t *to = a.packed + ((row * 2 + k) * a.inner + c0) / a.block * (a.block + 8);
                if (a.code == 0)
                    write_records<1, 0>(k ? u : g, col, left, to, a.block);
                else if (a.code == 1)
                    write_records<1, 1>(k ? u : g, col, left, to, a.block);
                else
                    write_records<1, 2>(k ? u : g, col, left, to, a.block);
            }
        }
    }
}

template <typename T>
cudaError_t gated(const GatedArgs &a, int sms, cudaStream_t stream)
{
    const T *x = static_cast<const T *>(a.x), *w = static_cast<const T *>(a.weight);
    float *z = static_cast<float *>(a.workspace);
    int64_t M = a.rows, N = 2 * a.inner, K = a.hidden;
    void *p[] = {&x, &w, &z, &M, &N, &K};
    cudaError_t e = launch_kernel(reinterpret_cast<void *>(&taco_gated_product_kernel<T, float, false>), 4 * sms, 256, 0, stream, p);
    if (e != cudaSuccess)
        return e;
    GatedArgs args = a;
    void *q[] = {&args, &z};
    return launch_kernel(a.activation == kSilu   ? reinterpret_cast<void *>(&taco_gated_finish_kernel<T, kSilu>)
                         : a.activation == kGelu ? reinterpret_cast<void *>(&taco_gated_finish_kernel<T, kGelu>)
                                                 : reinterpret_cast<void *>(&taco_gated_finish_kernel<T, kGeluTanh>),
                         8 * sms, 256, 0, stream, q);
}

template <typename T>
cudaError_t input_grad(const GatedInputGradArgs &a, int sms, cudaStream_t stream)
{
    const T *dz = static_cast<const T *>(a.dz), *w = static_cast<const T *>(a.weight);
    T *dx = static_cast<T *>(a.dx);
    int64_t M = a.rows, N = a.hidden, K = 2 * a.inner;
    void *p[] = {&dz, &w, &dx, &M, &N, &K};
    return launch_kernel(reinterpret_cast<void *>(&taco_gated_product_kernel<T, T, true>), 4 * sms, 256, 0, stream, p);
}

}  // namespace

cudaError_t init_gated() { return cudaSuccess; }

bool gated_in_range(int64_t rows, int64_t inner, int64_t hidden)
{
    // 32-bit coordinates, whole tiles past the end included
    return rows <= INT32_MAX - 256 && inner <= INT32_MAX / 2 - 256 && hidden <= INT32_MAX - 256;
}

int64_t gated_workspace(int64_t rows, int64_t inner, int64_t) { return 8 * rows * inner; }

int64_t gated_input_grad_workspace(int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_gated(const GatedArgs &a, uint32_t *, int sms, cudaStream_t stream)
{
    return a.dtype == kTypeBf16 ? gated<__nv_bfloat16>(a, sms, stream) : gated<__half>(a, sms, stream);
}

cudaError_t launch_gated_input_grad(const GatedInputGradArgs &a, uint32_t *, int sms, cudaStream_t stream)
{
    return a.dtype == kTypeBf16 ? input_grad<__nv_bfloat16>(a, sms, stream) : input_grad<__half>(a, sms, stream);
}

}  // namespace taco
