// taco_gated_grad.cu -- gradient of the gated product from the 8-bit checkpoint
// of its two projections, for GB300 (sm_103a).  Per element, with g = z_gate and
// u = z_up decoded from their records:
//   dz_gate = dy u act'(g),  dz_up = dy act(g),  y = act(g) u again,
// and the column sums of dz (the projections' bias gradients).
#include <algorithm>

#include "taco_activation.cuh"
#include "taco_kernels.h"

namespace taco {
namespace {

// A CTA takes a strip of `strip` vectors of eight columns (at most 32, strips of
// even size), a thread one of them, gate and up, in every 256 / strip-th row, so
// the bias gradients stay in its registers; the CTA's rows are added in order at
// the end.  The next row's loads are in flight.
// The sums take 32 registers: three CTAs an SM with them, four without.  8192 x 16384 bf16 SiLU with y again takes 207 us
// and with the sums 236; at 64 registers the sums spill (267), and 512 threads in two CTAs take 208 and 274.
constexpr int kThreads = 256;

template <typename T, int ACT, int CODE, bool SUMS>
__global__ void __launch_bounds__(kThreads, SUMS ? 3 : 4) taco_gated_grad_kernel(GatedGradArgs a, int strip)
{
    __shared__ float part[SUMS ? kThreads * 8 : 1];
    grid_launch_dependents();
    const int rows_a_pass = kThreads / strip, mine = threadIdx.x / strip, lane = threadIdx.x - mine * strip;
    const int64_t C = a.inner, col = (static_cast<int64_t>(blockIdx.x) * strip + lane) * 8;
    const bool in = mine < rows_a_pass && col < C;
    const int64_t step = static_cast<int64_t>(gridDim.y) * rows_a_pass;
    const int64_t block = col / a.block, half = C / a.block * (a.block + 8);   // half: record bytes of a row's gate
    const uint8_t *rec = a.packed + block * (a.block + 8);
    const int within = static_cast<int>(col - block * a.block);
    grid_dependency_wait();
    F8 sums[2] = {};
    Raw8<T> next_dy;
    uint2 next_codes[2] = {};
    float next_s[2] = {};
    auto fetch = [&](int64_t row) {
        if (in && row < a.rows) {
            next_dy = load_raw8(static_cast<const T *>(a.dy) + row * C + col);
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const uint8_t *r = rec + (2 * row + k) * half;
                next_codes[k] = *reinterpret_cast<const uint2 *>(r + within);
                next_s[k] = record_s(r, a.block);
            }
        }
    };
    int64_t row = static_cast<int64_t>(blockIdx.y) * rows_a_pass + mine;
    fetch(row);
    if (in)
        for (; row < a.rows; row += step) {
            const F8 dy = unpack(next_dy), qg = codes8_to_float(next_codes[0], CODE), qu = codes8_to_float(next_codes[1], CODE);
            const float sg = next_s[0], su = next_s[1];
            fetch(row + step);
            F8 dg, du, y;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float2 value, slope;
                activation_both2<ACT>(mul2(qg.v[i], both(sg)), value, slope);
                const float2 u = mul2(qu.v[i], both(su));
                dg.v[i] = mul2(mul2(dy.v[i], u), slope);
                du.v[i] = mul2(dy.v[i], value);
                y.v[i] = mul2(value, u);
                if (SUMS) {
                    sums[0].v[i] = add2(sums[0].v[i], dg.v[i]);
                    sums[1].v[i] = add2(sums[1].v[i], du.v[i]);
                }
            }
            T *dz = static_cast<T *>(a.dz) + row * 2 * C + col;
            store_raw8(dz, pack<T>(dg));
            store_raw8(dz + C, pack<T>(du));
            if (a.y)
                store_raw8(static_cast<T *>(a.y) + row * C + col, pack<T>(y));
        }
    if constexpr (SUMS) {
        // Sums of the rows that the CTA's threads took, column by column: the gate's, then the up projection's.
#pragma unroll
        for (int k = 0; k < 2; k++) {
            if (k)
                __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; i++) {
                part[2 * i * kThreads + threadIdx.x] = sums[k].v[i].x;
                part[(2 * i + 1) * kThreads + threadIdx.x] = sums[k].v[i].y;
            }
            __syncthreads();
            for (int c = threadIdx.x; c < strip * 8; c += kThreads) {
                const int64_t column = static_cast<int64_t>(blockIdx.x) * strip * 8 + c;
                if (column >= C)
                    break;
                float sum = 0.f;
                for (int r = 0; r < rows_a_pass; r++)
                    sum += part[(c & 7) * kThreads + r * strip + (c >> 3)];
                a.parts[static_cast<int64_t>(blockIdx.y) * 2 * C + k * C + column] = sum;
            }
        }
    }
}

template <typename T, int ACT, bool SUMS>
const void *kernel_of(int code)
{
    return code == 0   ? reinterpret_cast<void *>(&taco_gated_grad_kernel<T, ACT, 0, SUMS>)
           : code == 1 ? reinterpret_cast<void *>(&taco_gated_grad_kernel<T, ACT, 1, SUMS>)
                       : reinterpret_cast<void *>(&taco_gated_grad_kernel<T, ACT, 2, SUMS>);
}

template <typename T, bool SUMS>
const void *kernel_of(int activation, int code)
{
    return activation == kSilu   ? kernel_of<T, kSilu, SUMS>(code)
           : activation == kGelu ? kernel_of<T, kGelu, SUMS>(code)
                                 : kernel_of<T, kGeluTanh, SUMS>(code);
}

template <typename T>
const void *kernel_of(int activation, int code, bool sums)
{
    return sums ? kernel_of<T, true>(activation, code) : kernel_of<T, false>(activation, code);
}

}  // namespace

cudaError_t launch_gated_grad(int dtype, GatedGradArgs *a, int sms, cudaStream_t stream)
{
    const int64_t vectors = a->inner / 8, strips = (vectors + 31) / 32;
    int strip = static_cast<int>((vectors + strips - 1) / strips);
    const int64_t rows_a_pass = kThreads / strip, passes = (a->rows + rows_a_pass - 1) / rows_a_pass;
    a->nparts = static_cast<int>(std::min<int64_t>({passes, kMaxColumnParts, std::max<int64_t>(1, (a->parts ? 8 : 16) * sms / strips)}));
    void *p[] = {a, &strip};
    return launch_kernel_2d(dtype == kTypeBf16 ? kernel_of<__nv_bfloat16>(a->activation, a->code, a->parts) : kernel_of<__half>(a->activation, a->code, a->parts),
                            static_cast<unsigned>(strips), static_cast<unsigned>(a->nparts), kThreads, 0, stream, p);
}

}  // namespace taco
