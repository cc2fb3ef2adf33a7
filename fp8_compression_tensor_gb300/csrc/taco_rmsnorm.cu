// taco_rmsnorm.cu -- root-mean-square norm with the residual's addition, 8-bit
// checkpoints of the normalised rows and 8-bit outputs, for GB300 (sm_103a).
//
// Per row of C elements: h = x (or round(x + residual)),
//   rstd = 1 / sqrt(sum h^2 / C + eps),  xhat = h rstd,  y = xhat weight,
// y as a tensor or as records, and optionally the records of xhat
// (taco_train.cuh).  Sums are binary32.
#include "taco_norm.cuh"

namespace taco {
namespace {

// ---------------------------------------------------------------------------
// Any width: a CTA a row, element by element (no records: those need widths of
// whole blocks)
// ---------------------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(kRowThreads) taco_rms_any_kernel(RmsArgs a)
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
        float sq = 0.f;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            const float v = h(c);
            sq = fmaf(v, v, sq);
            if (res)
                static_cast<T *>(a.summed)[row * C + c] = from_float<T>(v);
        }
        const float rstd = inv_sqrt(cta_sum(sq, part) / static_cast<float>(C) + a.eps);
        if (threadIdx.x == 0)
            a.rstd[row] = rstd;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            float v = h(c) * rstd;
            if (a.weight)
                v *= load_param(a.weight, a.param_dtype, c);
            static_cast<T *>(a.y)[row * C + c] = from_float<T>(v);
        }
    }
}

// ---------------------------------------------------------------------------
// Widths of whole vectors of eight: a CTA a row, two vectors a lane at a time,
// the row read twice (the second time from L1 and L2)
// ---------------------------------------------------------------------------

constexpr int kWideThreads = 512;

template <int NV>
__device__ __forceinline__ void write_records_of(const F8 (&u)[NV], const int (&col)[NV], int C, uint8_t *row, int block, int code)
{
    if (code == 0)
        write_records<NV, 0>(u, col, C, row, block);
    else if (code == 1)
        write_records<NV, 1>(u, col, C, row, block);
    else
        write_records<NV, 2>(u, col, C, row, block);
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) taco_rms_wide_kernel(RmsArgs a)
{
    __shared__ float part[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * C;
        const T *res = a.residual ? static_cast<const T *>(a.residual) + row * C : nullptr;
        auto load = [&](int64_t c, bool store) {
            F8 h = unpack(load_raw8(x + c));
            if (res) {
                const F8 r = unpack(load_raw8(res + c));
#pragma unroll
                for (int i = 0; i < 4; i++)
                    h.v[i] = add2(h.v[i], r.v[i]);
                const Raw8<T> o = pack<T>(h);
                if (store)
                    store_raw8(static_cast<T *>(a.summed) + row * C + c, o);
                h = unpack(o);
            }
            return h;
        };
        float2 squares = both(0.f);
        for (int64_t base = warp * 512; base < C; base += kWideThreads * 16)
#pragma unroll
            for (int j = 0; j < 2; j++)
                if (base + j * 256 + lane * 8 < C) {
                    const F8 h = load(base + j * 256 + lane * 8, true);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        squares = fma2(h.v[i], h.v[i], squares);
                }
        const float rstd = inv_sqrt(cta_sum(squares.x + squares.y, part) / static_cast<float>(C) + a.eps);
        if (threadIdx.x == 0)
            a.rstd[row] = rstd;
        for (int64_t base = warp * 512; base < C; base += kWideThreads * 16) {
            F8 h[2] = {}, y[2] = {};
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int64_t c = base + j * 256 + lane * 8;
                if (c < C) {
                    h[j] = load(c, false);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        y[j].v[i] = h[j].v[i] = mul2(h[j].v[i], both(rstd));
                    if (a.weight) {
                        const F8 w = load_param_f8(a.weight, a.param_dtype, c);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            y[j].v[i] = mul2(y[j].v[i], w.v[i]);
                    }
                    if (a.y)
                        store_raw8(static_cast<T *>(a.y) + row * C + c, pack<T>(y[j]));
                }
            }
            const int left = static_cast<int>(C - base < 512 ? C - base : 512), col[2] = {lane * 8, 256 + lane * 8};
            if (a.packed)
                write_records_of<2>(h, col, left, a.packed + (row * C + base) / a.block * (a.block + 8), a.block, a.code);
            if (a.packed_y)
                write_records_of<2>(y, col, left, a.packed_y + (row * C + base) / a.block * (a.block + 8), a.block, a.code);
        }
    }
}

template <typename T>
cudaError_t rms_any(const RmsArgs &a, int sms, cudaStream_t stream)
{
    RmsArgs args = a;
    void *p[] = {&args};
    if (a.hidden % 8 == 0)
        return launch_kernel(reinterpret_cast<void *>(&taco_rms_wide_kernel<T>), row_grid(a.rows, sms, 4), kWideThreads, 0, stream, p);
    return launch_kernel(reinterpret_cast<void *>(&taco_rms_any_kernel<T>), row_grid(a.rows, sms, 8), kRowThreads, 0, stream, p);
}

}  // namespace

cudaError_t init_rms() { return cudaSuccess; }

cudaError_t launch_rms(int dtype, const RmsArgs &a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? rms_any<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? rms_any<__half>(a, sms, stream)
                               : rms_any<float>(a, sms, stream);
}

}  // namespace taco
