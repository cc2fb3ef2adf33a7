// taco_layernorm.cu -- layer norm, forward and backward, with 8-bit
// checkpoints of the normalised input, for GB300 (sm_103a).
//
// Forward, per row of C elements: h = x (or round(x + residual)),
//   mu = sum h / C,  v = sum (h - mu)^2 / C,  rstd = 1 / sqrt(v + eps),
//   xhat = (h - mu) rstd,  y = xhat weight + bias,
// and optionally the records of xhat (taco_train.cuh).  Statistics are
// binary32, the variance from the centred values (a second pass), so a large
// mean costs no precision.
//
// Backward, with a = dy weight:
//   c1 = sum a / C,  c2 = sum a xhat / C,  dx = rstd (a - c1 - xhat c2) [+ dsummed],
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy,
// xhat from (x, mean, rstd) or from records.
#include "taco_kernels.h"
#include "taco_train.cuh"

namespace taco {
namespace {

constexpr int kRowThreads = 256;

// ---------------------------------------------------------------------------
// Any width: one CTA per row, element by element
// ---------------------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(kRowThreads) taco_norm_any_kernel(NormArgs a)
{
    __shared__ float part[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * C;
        const T *res = a.residual ? static_cast<const T *>(a.residual) + row * C : nullptr;
        auto h = [&](int64_t c) {
            const float v = to_float(x[c]);
            return res ? to_float(from_float<T>(v + to_float(res[c]))) : v;
        };
        float sum = 0.f;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            const float v = h(c);
            sum += v;
            if (res)
                static_cast<T *>(a.summed)[row * C + c] = from_float<T>(v);
        }
        const float mean = cta_sum(sum, part) / static_cast<float>(C);
        float sq = 0.f;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            const float d = h(c) - mean;
            sq = fmaf(d, d, sq);
        }
        const float rstd = 1.f / sqrtf(cta_sum(sq, part) / static_cast<float>(C) + a.eps);
        if (threadIdx.x == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            float v = (h(c) - mean) * rstd;
            if (a.weight)
                v *= load_param(a.weight, a.param_dtype, c);
            if (a.bias)
                v += load_param(a.bias, a.param_dtype, c);
            static_cast<T *>(a.y)[row * C + c] = from_float<T>(v);
        }
        if (!a.packed)
            continue;
        // Records: a warp per block.
        const int lane = threadIdx.x & 31, B = a.block;
        for (int64_t k = threadIdx.x >> 5; k < C / B; k += kRowThreads / 32) {
            uint32_t top = 0;
            for (int i = lane; i < B; i += 32)
                top = max(top, abs_bits((h(k * B + i) - mean) * rstd));
            top = __reduce_max_sync(kFullMask, top);
            float inv;
            const float s = record_scale(top, a.code, &inv);
            uint8_t *rec = a.packed + (row * (C / B) + k) * (B + 8);
            for (int i = lane; i < B; i += 32)
                rec[i] = record_code((h(k * B + i) - mean) * rstd, inv, a.code);
            if (lane == 0)
                *reinterpret_cast<float2 *>(rec + B) = make_float2(1.f, s);
        }
    }
}

// dx of any width: one CTA per row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) taco_norm_grad_any_kernel(NormGradArgs a)
{
    __shared__ float part[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *dy = static_cast<const T *>(a.dy) + row * C;
        const float rstd = a.rstd[row], mean = a.x ? a.mean[row] : 0.f;
        auto xhat = [&](int64_t c) {
            return a.x ? (to_float(static_cast<const T *>(a.x)[row * C + c]) - mean) * rstd
                       : record_value(a.packed, row * C + c, a.block, a.code);
        };
        auto grad = [&](int64_t c) {
            const float v = to_float(dy[c]);
            return a.weight ? v * load_param(a.weight, a.param_dtype, c) : v;
        };
        float s1 = 0.f, s2 = 0.f;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            const float g = grad(c);
            s1 += g;
            s2 = fmaf(g, xhat(c), s2);
        }
        const float c1 = cta_sum(s1, part) / static_cast<float>(C), c2 = cta_sum(s2, part) / static_cast<float>(C);
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            float v = rstd * (grad(c) - c1 - xhat(c) * c2);
            if (a.dsummed)
                v += to_float(static_cast<const T *>(a.dsummed)[row * C + c]);
            static_cast<T *>(a.dx)[row * C + c] = from_float<T>(v);
        }
    }
}

// Column sums of dy xhat and dy over the rows part, part + nparts, ...: a
// thread per column.
template <typename T>
__global__ void __launch_bounds__(128) taco_norm_grad_columns_kernel(NormGradArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden, c = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (c >= C)
        return;
    float dw = 0.f, db = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += a.nparts) {
        const float g = to_float(static_cast<const T *>(a.dy)[row * C + c]);
        const float xh = a.x ? (to_float(static_cast<const T *>(a.x)[row * C + c]) - a.mean[row]) * a.rstd[row]
                             : record_value(a.packed, row * C + c, a.block, a.code);
        dw = fmaf(g, xh, dw);
        db += g;
    }
    a.parts[static_cast<int64_t>(blockIdx.y) * C + c] = dw;
    a.parts[static_cast<int64_t>(a.nparts + blockIdx.y) * C + c] = db;
}

// out[c] = sum over p of parts[p][c]: a warp's lanes take 32 columns, the
// CTA's eight warps every eighth p, and the eight sums are added in order.
__global__ void __launch_bounds__(256) taco_column_sums_kernel(const float *parts, int nparts, int64_t n, void *out,
                                                               void *out2, int dtype)
{
    __shared__ float part[8][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    void *to = blockIdx.y ? out2 : out;
    if (!to)
        return;
    const float *p = parts + static_cast<int64_t>(blockIdx.y) * nparts * n;
    float sum = 0.f;
    if (c < n)
        for (int i = warp; i < nparts; i += 8)
            sum += p[static_cast<int64_t>(i) * n + c];
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < n) {
        for (int w = 1; w < 8; w++)
            sum += part[w][lane];
        store_param(to, dtype, c, sum);
    }
}

int row_grid(int64_t rows, int sms, int per_sm)
{
    const int64_t cap = static_cast<int64_t>(sms) * per_sm;
    return static_cast<int>(rows < cap ? rows : cap);
}

template <typename T>
cudaError_t norm_any(const NormArgs &a, int sms, cudaStream_t stream)
{
    NormArgs args = a;
    void *p[] = {&args};
    return launch_kernel(reinterpret_cast<void *>(&taco_norm_any_kernel<T>), row_grid(a.rows, sms, 8), kRowThreads, 0,
                         stream, p);
}

template <typename T>
cudaError_t norm_grad_any(const NormGradArgs &a, int sms, cudaStream_t stream)
{
    NormGradArgs args = a;
    void *p[] = {&args};
    cudaError_t e = launch_kernel(reinterpret_cast<void *>(&taco_norm_grad_any_kernel<T>), row_grid(a.rows, sms, 8),
                                  kRowThreads, 0, stream, p);
    if (e == cudaSuccess && a.parts)
        e = launch_kernel_2d(reinterpret_cast<void *>(&taco_norm_grad_columns_kernel<T>),
                             static_cast<unsigned>((a.hidden + 127) / 128), static_cast<unsigned>(a.nparts), 128, 0, stream, p);
    return e;
}

}  // namespace

cudaError_t launch_column_sums(const float *parts, int nparts, int64_t n, void *out, void *out2, int dtype,
                               cudaStream_t stream)
{
    void *p[] = {&parts, &nparts, &n, &out, &out2, &dtype};
    return launch_kernel_2d(reinterpret_cast<void *>(&taco_column_sums_kernel), static_cast<unsigned>((n + 31) / 32),
                            out2 ? 2u : 1u, 256, 0, stream, p);
}

cudaError_t launch_norm(int dtype, const NormArgs &a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? norm_any<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? norm_any<__half>(a, sms, stream)
                               : norm_any<float>(a, sms, stream);
}

cudaError_t launch_norm_grad(int dtype, NormGradArgs *a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? norm_grad_any<__nv_bfloat16>(*a, sms, stream)
           : dtype == kTypeF16 ? norm_grad_any<__half>(*a, sms, stream)
                               : norm_grad_any<float>(*a, sms, stream);
}

}  // namespace taco
