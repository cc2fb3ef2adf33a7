// taco_rmsnorm_grad.cu -- gradients of the root-mean-square norm, from its input
// or from 8-bit checkpoints, for GB300 (sm_103a).  With a = dy weight:
//   c = sum a xhat / C,  dx = rstd (a - xhat c) [+ dsummed],
//   dweight = sum over rows of dy xhat,
// xhat = x rstd, or from records.
#include "taco_norm.cuh"

namespace taco {
namespace {

// ---------------------------------------------------------------------------
// Any width: dx with a CTA a row, element by element, and the column sums in a
// pass of their own
// ---------------------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(kRowThreads) taco_rms_grad_any_kernel(RmsGradArgs a)
{
    __shared__ float part[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row];
        auto xhat = [&](int64_t c) { return to_float(static_cast<const T *>(a.x)[row * C + c]) * rstd; };
        auto grad = [&](int64_t c) {
            const float v = to_float(static_cast<const T *>(a.dy)[row * C + c]);
            return a.weight ? v * load_param(a.weight, a.param_dtype, c) : v;
        };
        float s = 0.f;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads)
            s = fmaf(grad(c), xhat(c), s);
        const float mean = cta_sum(s, part) / static_cast<float>(C);
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            float v = rstd * fmaf(-xhat(c), mean, grad(c));
            if (a.dsummed)
                v += to_float(static_cast<const T *>(a.dsummed)[row * C + c]);
            static_cast<T *>(a.dx)[row * C + c] = from_float<T>(v);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(128) taco_rms_grad_columns_kernel(RmsGradArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden, c = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (c >= C)
        return;
    float dw = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += a.nparts)
        dw = fmaf(to_float(static_cast<const T *>(a.dy)[row * C + c]),
                  to_float(static_cast<const T *>(a.x)[row * C + c]) * a.rstd[row], dw);
    a.parts[static_cast<int64_t>(blockIdx.y) * C + c] = dw;
}

// ---------------------------------------------------------------------------
// Widths of whole vectors of eight
// ---------------------------------------------------------------------------

// xhat of eight columns from c on.
template <typename T>
__device__ __forceinline__ F8 load_normalised(const RmsGradArgs &a, int64_t row, int64_t c, float rstd)
{
    F8 f;
    float s = rstd;
    if (a.x) {
        f = unpack(load_raw8(static_cast<const T *>(a.x) + row * a.hidden + c));
    } else {
        const int64_t k = (row * a.hidden + c) / a.block;
        const uint8_t *rec = a.packed + k * (a.block + 8);
        f = codes8_to_float(*reinterpret_cast<const uint2 *>(rec + (row * a.hidden + c - k * a.block)), a.code);
        s = record_s(rec, a.block);
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
        f.v[i] = mul2(f.v[i], both(s));
    return f;
}

// dx with a CTA a row, read twice.
constexpr int kWideThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kWideThreads) taco_rms_grad_wide_kernel(RmsGradArgs a)
{
    __shared__ float part[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row];
        auto weighted = [&](int64_t c) {
            F8 g = unpack(load_raw8(static_cast<const T *>(a.dy) + row * C + c));
            if (a.weight) {
                const F8 w = load_param_f8(a.weight, a.param_dtype, c);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    g.v[i] = mul2(g.v[i], w.v[i]);
            }
            return g;
        };
        float2 t = both(0.f);
        for (int64_t c = threadIdx.x * 8; c < C; c += kWideThreads * 8) {
            const F8 w = weighted(c), xh = load_normalised<T>(a, row, c, rstd);
#pragma unroll
            for (int i = 0; i < 4; i++)
                t = fma2(w.v[i], xh.v[i], t);
        }
        const float mean = cta_sum(t.x + t.y, part) / static_cast<float>(C);
        for (int64_t c = threadIdx.x * 8; c < C; c += kWideThreads * 8) {
            F8 w = weighted(c);
            const F8 xh = load_normalised<T>(a, row, c, rstd);
#pragma unroll
            for (int i = 0; i < 4; i++)
                w.v[i] = mul2(fma2(xh.v[i], both(-mean), w.v[i]), both(rstd));
            if (a.dsummed) {
                const F8 s = unpack(load_raw8(static_cast<const T *>(a.dsummed) + row * C + c));
#pragma unroll
                for (int i = 0; i < 4; i++)
                    w.v[i] = add2(w.v[i], s.v[i]);
            }
            store_raw8(static_cast<T *>(a.dx) + row * C + c, pack<T>(w));
        }
    }
}

// Column sums over the rows part, part + nparts, ...: eight columns a thread.
template <typename T>
__global__ void __launch_bounds__(128) taco_rms_grad_wide_columns_kernel(RmsGradArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden, c = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) * 8;
    if (c >= C)
        return;
    F8 dw = {};
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < a.rows; row += a.nparts) {
        const F8 g = unpack(load_raw8(static_cast<const T *>(a.dy) + row * C + c)), xh = load_normalised<T>(a, row, c, a.rstd[row]);
#pragma unroll
        for (int i = 0; i < 4; i++)
            dw.v[i] = fma2(g.v[i], xh.v[i], dw.v[i]);
    }
    store_raw8(a.parts + static_cast<int64_t>(blockIdx.y) * C + c, pack<float>(dw));
}

template <typename T>
cudaError_t rms_grad_any(RmsGradArgs *a, int sms, cudaStream_t stream)
{
    void *p[] = {a};
    const bool vectors = a->hidden % 8 == 0;
    // about eight CTAs of 128 threads an SM for the column sums
    const int64_t across = vectors ? (a->hidden + 1023) / 1024 : (a->hidden + 127) / 128;
    a->nparts = static_cast<int>(std::min<int64_t>({a->rows, kMaxColumnParts, std::max<int64_t>(1, 8 * sms / across)}));
    cudaError_t e = vectors ? launch_kernel(reinterpret_cast<void *>(&taco_rms_grad_wide_kernel<T>), row_grid(a->rows, sms, 4),
                                            kWideThreads, 0, stream, p)
                            : launch_kernel(reinterpret_cast<void *>(&taco_rms_grad_any_kernel<T>), row_grid(a->rows, sms, 8),
                                            kRowThreads, 0, stream, p);
    if (e == cudaSuccess && a->parts)
        e = launch_kernel_2d(vectors ? reinterpret_cast<void *>(&taco_rms_grad_wide_columns_kernel<T>)
                                     : reinterpret_cast<void *>(&taco_rms_grad_columns_kernel<T>),
                             static_cast<unsigned>(across), static_cast<unsigned>(a->nparts), 128, 0, stream, p);
    return e;
}

}  // namespace

cudaError_t init_rms_grad() { return cudaSuccess; }

cudaError_t launch_rms_grad(int dtype, RmsGradArgs *a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? rms_grad_any<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? rms_grad_any<__half>(a, sms, stream)
                               : rms_grad_any<float>(a, sms, stream);
}

}  // namespace taco
