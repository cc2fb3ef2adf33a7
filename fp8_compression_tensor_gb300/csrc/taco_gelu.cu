// taco_gelu.cu -- GELU with an 8-bit checkpoint of its input, and its backward
// pass from that checkpoint, for GB300 (sm_103a).
//
// Forward: u = x + bias (binary32), y = u Phi(u) with the normal distribution
// function Phi, or the tanh form y = u/2 (1 + tanh(a (u + b u^3))), a =
// sqrt(2/pi), b = 0.044715; the records of u (taco_train.cuh).
//
// Backward, with u decoded from the records: dx = dy (Phi(u) + u phi(u)), or
// the tanh form's slope; dbias = sum over rows of dx; y again when the next
// weight gradient needs it.
#include "taco_kernels.h"
#include "taco_train.cuh"

namespace taco {
namespace {

constexpr float kTanhA = 0.7978845608028654f, kTanhB = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f, kInvSqrt2Pi = 0.3989422804014327f;

// Phi(u) from the complementary error function: no cancellation for negative u.
__device__ __forceinline__ float normal_cdf(float u) { return 0.5f * erfcf(-kSqrtHalf * u); }

__device__ __forceinline__ float gelu_value(float u, int tanh_form)
{
    if (tanh_form)
        return 0.5f * u * (1.f + tanhf(kTanhA * (u + kTanhB * u * u * u)));
    return u * normal_cdf(u);
}

__device__ __forceinline__ float gelu_slope(float u, int tanh_form)
{
    if (tanh_form) {
        const float t = tanhf(kTanhA * (u + kTanhB * u * u * u));
        return 0.5f * (1.f + t) + 0.5f * u * (1.f - t * t) * kTanhA * (1.f + 3.f * kTanhB * u * u);
    }
    return normal_cdf(u) + u * kInvSqrt2Pi * expf(-0.5f * u * u);
}

// A warp per block of B elements (without records: any pieces of B elements, the last one ragged).
template <typename T>
__global__ void __launch_bounds__(256) taco_gelu_kernel(GeluArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, B = a.block;
    const int64_t n = a.rows * a.hidden, blocks = (n + B - 1) / B;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); k < blocks; k += 8ll * gridDim.x) {
        const int len = static_cast<int>(n - k * B < B ? n - k * B : B);
        float u[16];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const int i = lane + 32 * j;
            if (i < len) {
                u[j] = to_float(static_cast<const T *>(a.x)[k * B + i]);
                if (a.bias)
                    u[j] += load_param(a.bias, a.param_dtype, (k * B + i) % a.hidden);
                top = max(top, abs_bits(u[j]));
            }
        }
        float inv = 0.f, s = 0.f;
        uint8_t *rec = a.packed + k * (B + 8);
        if (a.packed) {
            top = __reduce_max_sync(kFullMask, top);
            s = record_scale(top, a.code, &inv);
            if (lane == 0)
                *reinterpret_cast<float2 *>(rec + B) = make_float2(1.f, s);
        }
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const int i = lane + 32 * j;
            if (i < len) {
                static_cast<T *>(a.y)[k * B + i] = from_float<T>(gelu_value(u[j], a.tanh_form));
                if (a.packed)
                    rec[i] = record_code(u[j], inv, a.code);
            }
        }
    }
}

// A thread per column, rows part, part + nparts, ...
template <typename T>
__global__ void __launch_bounds__(128) taco_gelu_grad_kernel(GeluGradArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden, c = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (c >= C)
        return;
    float db = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += a.nparts) {
        const int64_t i = row * C + c;
        const float u = record_value(a.packed, i, a.block, a.code);
        const float d = to_float(static_cast<const T *>(a.dy)[i]) * gelu_slope(u, a.tanh_form);
        static_cast<T *>(a.dx)[i] = from_float<T>(d);
        if (a.y)
            static_cast<T *>(a.y)[i] = from_float<T>(gelu_value(u, a.tanh_form));
        db += d;
    }
    if (a.parts)
        a.parts[static_cast<int64_t>(blockIdx.y) * C + c] = db;
}

template <typename T>
cudaError_t gelu(const GeluArgs &a, int sms, cudaStream_t stream)
{
    GeluArgs args = a;
    if (!a.packed)
        args.block = 512;
    void *p[] = {&args};
    const int64_t want = (a.rows * a.hidden + 8ll * args.block - 1) / (8ll * args.block), cap = static_cast<int64_t>(sms) * 32;
    return launch_kernel(reinterpret_cast<void *>(&taco_gelu_kernel<T>), static_cast<int>(want < cap ? want : cap), 256,
                         0, stream, p);
}

template <typename T>
cudaError_t gelu_grad(const GeluGradArgs &a, int, cudaStream_t stream)
{
    GeluGradArgs args = a;
    void *p[] = {&args};
    return launch_kernel_2d(reinterpret_cast<void *>(&taco_gelu_grad_kernel<T>),
                            static_cast<unsigned>((a.hidden + 127) / 128), static_cast<unsigned>(a.nparts), 128, 0, stream, p);
}

}  // namespace

cudaError_t launch_gelu(int dtype, const GeluArgs &a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? gelu<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? gelu<__half>(a, sms, stream)
                               : gelu<float>(a, sms, stream);
}

cudaError_t launch_gelu_grad(int dtype, GeluGradArgs *a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? gelu_grad<__nv_bfloat16>(*a, sms, stream)
           : dtype == kTypeF16 ? gelu_grad<__half>(*a, sms, stream)
                               : gelu_grad<float>(*a, sms, stream);
}

}  // namespace taco
