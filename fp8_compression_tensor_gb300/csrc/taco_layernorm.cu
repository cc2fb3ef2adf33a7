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
#include <algorithm>

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

// ---------------------------------------------------------------------------
// Widths of whole vectors of eight: rows in registers
// ---------------------------------------------------------------------------

__device__ __forceinline__ void group_barrier(int id, int threads)
{
    asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sum over the `warps` warps of a row group, the same for all its threads.
// `part` is the group's own; the caller alternates between two of them, so one
// barrier a sum is enough: a thread writes a part again only behind the next
// sum's barrier, when every thread has read it.
__device__ __forceinline__ float group_sum(float v, float *part, int warp, int warps, int barrier_id)
{
    v = warp_sum(v);
    if (warps == 1)
        return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0)
        part[warp] = v;
    group_barrier(barrier_id, warps * 32);
    return warp_sum(lane < warps ? part[lane] : 0.f);
}

// 1 / sqrt(v): the hardware's estimate and one Newton step.
__device__ __forceinline__ float inv_sqrt(float v)
{
    const float r = rsqrtf(v);
    return v > 0.f && v < 3.0e38f ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
}

constexpr int kNormThreads = 1024;
constexpr int kGradThreads = 512;

// A group of `warps` warps holds a row in registers: NV vectors of eight
// elements a lane, vector j of warp w from column 256 (w NV + j) on.  The CTA's
// groups take rows in turn; weight and bias are read from global memory once,
// into shared memory (STAGED; with one row a group, straight from global
// memory), and the next row's loads are in flight while this row is reduced.
template <typename T, int NV, bool STAGED>
__global__ void __launch_bounds__(kNormThreads, 1) taco_norm_kernel(NormArgs a, int warps, int groups)
{
    extern __shared__ float sparam[];              // weight, then bias, `hidden` each (STAGED)
    __shared__ float parts[2][32];
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int C = static_cast<int>(a.hidden);
    float *part0 = parts[0] + group * warps, *part1 = parts[1] + group * warps;
    const float inv_c = 1.f / static_cast<float>(C);
    int col[NV];
#pragma unroll
    for (int j = 0; j < NV; j++)
        col[j] = ((warp * NV + j) * 32 + lane) * 8;
    grid_dependency_wait();
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    Raw8<T> nx[NV], nr[NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (r < a.rows && col[j] < C) {
                nx[j] = load_raw8(x + r * C + col[j]);
                if (res)
                    nr[j] = load_raw8(res + r * C + col[j]);
            }
    };
    fetch(row);
    if (STAGED) {
        for (int c = threadIdx.x * 8; c < C; c += blockDim.x * 8) {
            float f[8];
            if (a.weight) {
                load_param8(a.weight, a.param_dtype, c, f);
                for (int i = 0; i < 8; i++)
                    sparam[c + i] = f[i];
            }
            if (a.bias) {
                load_param8(a.bias, a.param_dtype, c, f);
                for (int i = 0; i < 8; i++)
                    sparam[C + c + i] = f[i];
            }
        }
        __syncthreads();
    }
    for (; row < a.rows; row += step) {
        float h[NV][8];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; j++) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                h[j][i] = 0.f;
            if (col[j] < C) {
                unpack8(nx[j], h[j]);
                if (res) {
                    float r[8];
                    unpack8(nr[j], r);
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        h[j][i] += r[i];
                    const Raw8<T> o = pack8(h[j], x);
#pragma unroll
                    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); i++)
                        reinterpret_cast<uint4 *>(static_cast<T *>(a.summed) + row * C + col[j])[i] = o.v[i];
                    unpack8(o, h[j]);
                }
#pragma unroll
                for (int i = 0; i < 8; i++)
                    sum += h[j][i];
            }
        }
        fetch(row + step);
        const float mean = group_sum(sum, part0, warp, warps, 1 + group) / static_cast<float>(C);   // exact for constant rows
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (col[j] < C) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    h[j][i] -= mean;
                    sq = fmaf(h[j][i], h[j][i], sq);
                }
            }
        const float rstd = inv_sqrt(fmaf(group_sum(sq, part1, warp, warps, 1 + group), inv_c, a.eps));
        if (warp == 0 && lane == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (col[j] < C) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; i++)
                    y[i] = h[j][i] *= rstd;
                if (a.weight) {
                    float w[8];
                    if (STAGED)
                        unpack8(Raw8<float>{{*reinterpret_cast<const uint4 *>(sparam + col[j]),
                                             *reinterpret_cast<const uint4 *>(sparam + col[j] + 4)}}, w);
                    else
                        load_param8(a.weight, a.param_dtype, col[j], w);
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        y[i] *= w[i];
                }
                if (a.bias) {
                    float b[8];
                    if (STAGED)
                        unpack8(Raw8<float>{{*reinterpret_cast<const uint4 *>(sparam + C + col[j]),
                                             *reinterpret_cast<const uint4 *>(sparam + C + col[j] + 4)}}, b);
                    else
                        load_param8(a.bias, a.param_dtype, col[j], b);
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        y[i] += b[i];
                }
                store8(static_cast<T *>(a.y) + row * C + col[j], y);
            }
        if (a.packed) {
            uint8_t *at[NV];
            const int64_t pitch = record_offset(C, a.block);
#pragma unroll
            for (int j = 0; j < NV; j++)
                at[j] = col[j] < C ? a.packed + row * pitch + record_offset(col[j], a.block) : nullptr;
            write_records<NV>(h, at, a.block, a.code);
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

// Rows of whole vectors, the same layout of a row over a group of warps as the
// forward pass, so a thread keeps its columns and adds up their dweight and
// dbias in registers over all rows that its group takes.  Each thread copies its
// own pieces of the next rows (dy, x, dsummed) to shared memory with cp.async,
// `stages` rows deep, and reads only what it copied itself, so the copies need
// no barrier; a row's two sums need one.  Codes and scales of records, 8 bytes
// each, are loaded to registers a row ahead.
template <typename T, int NV, bool RECORDS>
__global__ void __launch_bounds__(kGradThreads, 1)
taco_norm_grad_kernel(NormGradArgs a, int warps, int groups, int stages)
{
    extern __shared__ __align__(16) uint8_t dynamic[];
    __shared__ float2 parts[2][32];
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int C = static_cast<int>(a.hidden), nthreads = blockDim.x;
    constexpr int kUnits = sizeof(T) / 2;            // 16-byte units of eight elements
    const int per_stage = (1 + !RECORDS + (a.dsummed != nullptr)) * NV * kUnits;
    float *sweight = reinterpret_cast<float *>(dynamic);
    uint4 *ring = reinterpret_cast<uint4 *>(dynamic + (a.weight ? (C * 4 + 15) / 16 * 16 : 0));
    const uint32_t ring_at = smem_addr(ring) + threadIdx.x * 16;
    int col[NV];
    int64_t rec[NV], meta[NV];
#pragma unroll
    for (int j = 0; j < NV; j++) {
        col[j] = ((warp * NV + j) * 32 + lane) * 8;
        if (RECORDS) {
            rec[j] = record_offset(col[j], a.block);
            meta[j] = static_cast<int64_t>(col[j] / a.block) * (a.block + 8) + a.block;
        }
    }
    const int64_t pitch = RECORDS ? record_offset(C, a.block) : 0;
    grid_dependency_wait();
    if (a.weight) {
        for (int c = threadIdx.x * 8; c < C; c += nthreads * 8) {
            float f[8];
            load_param8(a.weight, a.param_dtype, c, f);
            for (int i = 0; i < 8; i++)
                sweight[c + i] = f[i];
        }
        __syncthreads();
    }
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group, step = static_cast<int64_t>(gridDim.x) * groups;
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            uint32_t to = ring_at + static_cast<uint32_t>(stage * per_stage * nthreads) * 16u;
            auto piece = [&](const void *src) {
#pragma unroll
                for (int j = 0; j < NV; j++)
#pragma unroll
                    for (int k = 0; k < kUnits; k++, to += nthreads * 16)
                        if (col[j] < C)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to),
                                         "l"(reinterpret_cast<const uint4 *>(static_cast<const T *>(src) + row * C + col[j]) + k)
                                         : "memory");
            };
            piece(a.dy);
            if (!RECORDS)
                piece(a.x);
            if (a.dsummed)
                piece(a.dsummed);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint2 codes[NV], scales[NV];
    float next_rstd = 0.f, next_mean = 0.f;
    auto fetch = [&](int64_t row) {
        if (row >= a.rows)
            return;
        next_rstd = __ldg(a.rstd + row);
        if (!RECORDS)
            next_mean = __ldg(a.mean + row);
        if (RECORDS) {
#pragma unroll
            for (int j = 0; j < NV; j++)
                if (col[j] < C) {
                    codes[j] = __ldg(reinterpret_cast<const uint2 *>(a.packed + row * pitch + rec[j]));
                    scales[j] = __ldg(reinterpret_cast<const uint2 *>(a.packed + row * pitch + meta[j]));
                }
        }
    };
    float dw[NV][8], db[NV][8];
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
        for (int i = 0; i < 8; i++)
            dw[j][i] = db[j][i] = 0.f;
    for (int i = 0; i < stages - 1; i++)
        copy_row(first + i * step, i);
    fetch(first);
    int stage = 0, fill = stages - 1;
    uint32_t side = 0;
    for (int64_t row = first; row < a.rows; row += step, side ^= 1u) {
        copy_row(row + (stages - 1) * step, fill);
        fill = fill + 1 == stages ? 0 : fill + 1;
        if (stages == 4)
            asm volatile("cp.async.wait_group 3;" ::: "memory");
        else if (stages == 3)
            asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (stages == 2)
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        const uint4 *mine = ring + threadIdx.x + static_cast<size_t>(stage) * per_stage * nthreads;
        stage = stage + 1 == stages ? 0 : stage + 1;
        const float rstd = next_rstd, mean = next_mean;
        uint2 q[NV];
        float factor[NV];
        if (RECORDS) {
#pragma unroll
            for (int j = 0; j < NV; j++) {
                q[j] = codes[j];
                factor[j] = meta_factor(scales[j]);
            }
        }
        fetch(row + step);
        // Vector j of the thread's piece `tensor`, and xhat of vector j.
        auto vector = [&](int tensor, int j, float (&f)[8]) {
            Raw8<T> r;
#pragma unroll
            for (int k = 0; k < kUnits; k++)
                r.v[k] = mine[static_cast<size_t>((tensor * NV + j) * kUnits + k) * nthreads];
            unpack8(r, f);
        };
        auto normalised = [&](int j, float (&f)[8]) {
            if (RECORDS) {
                codes8_to_float(q[j], a.code, f);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    f[i] *= factor[j];
            } else {
                vector(1, j, f);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    f[i] = (f[i] - mean) * rstd;
            }
        };
        auto weighted = [&](int j, const float (&g)[8], float (&f)[8]) {
            if (a.weight) {
                const float4 lo = *reinterpret_cast<const float4 *>(sweight + col[j]), hi = *reinterpret_cast<const float4 *>(sweight + col[j] + 4);
                f[0] = g[0] * lo.x, f[1] = g[1] * lo.y, f[2] = g[2] * lo.z, f[3] = g[3] * lo.w;
                f[4] = g[4] * hi.x, f[5] = g[5] * hi.y, f[6] = g[6] * hi.z, f[7] = g[7] * hi.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    f[i] = g[i];
            }
        };
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (col[j] < C) {
                float g[8], xh[8], w[8];
                vector(0, j, g);
                normalised(j, xh);
                weighted(j, g, w);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    s1 += w[i];
                    s2 = fmaf(w[i], xh[i], s2);
                }
            }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (warps > 1) {
            float2 *part = parts[side] + group * warps;
            if (lane == 0)
                part[warp] = make_float2(s1, s2);
            group_barrier(1 + group, warps * 32);
            const float2 v = lane < warps ? part[lane] : make_float2(0.f, 0.f);
            s1 = warp_sum(v.x);
            s2 = warp_sum(v.y);
        }
        const float c1 = s1 / static_cast<float>(C), c2 = s2 / static_cast<float>(C);
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (col[j] < C) {
                float g[8], xh[8], w[8];
                vector(0, j, g);
                normalised(j, xh);
                weighted(j, g, w);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    dw[j][i] = fmaf(g[i], xh[i], dw[j][i]);
                    db[j][i] += g[i];
                    w[i] = rstd * fmaf(-xh[i], c2, w[i] - c1);
                }
                if (a.dsummed) {
                    vector(RECORDS ? 1 : 2, j, g);
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        w[i] += g[i];
                }
                store8(static_cast<T *>(a.dx) + row * C + col[j], w);
            }
    }
    if (!a.parts)
        return;
    // The groups' sums, added in order in the ring's place.
    float *sums = reinterpret_cast<float *>(ring);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (int g = 0; g < groups; g++) {
        __syncthreads();
        if (g == group) {
#pragma unroll
            for (int j = 0; j < NV; j++)
                if (col[j] < C) {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        if (g > 0) {
                            dw[j][i] += sums[(i * 2) * (C / 8) + col[j] / 8];
                            db[j][i] += sums[(i * 2 + 1) * (C / 8) + col[j] / 8];
                        }
                        if (g + 1 < groups) {
                            sums[(i * 2) * (C / 8) + col[j] / 8] = dw[j][i];
                            sums[(i * 2 + 1) * (C / 8) + col[j] / 8] = db[j][i];
                        }
                    }
                    if (g + 1 == groups) {
                        store8(a.parts + static_cast<int64_t>(blockIdx.x) * C + col[j], dw[j]);
                        store8(a.parts + static_cast<int64_t>(a.nparts + blockIdx.x) * C + col[j], db[j]);
                    }
                }
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
// CTA's 32 warps every 32nd p, and the 32 sums are added in order.
__global__ void __launch_bounds__(1024) taco_column_sums_kernel(const float *parts, int nparts, int64_t n, void *out,
                                                               void *out2, int dtype)
{
    __shared__ float part[32][32];
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
        #pragma unroll 4
        for (int i = warp; i < nparts; i += 32)
            sum += p[static_cast<int64_t>(i) * n + c];
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < n) {
        for (int w = 1; w < 32; w++)
            sum += part[w][lane];
        store_param(to, dtype, c, sum);
    }
}

int row_grid(int64_t rows, int sms, int per_sm)
{
    const int64_t cap = static_cast<int64_t>(sms) * per_sm;
    return static_cast<int>(rows < cap ? rows : cap);
}

// Whole vectors of eight, and at most 32 warps of two vectors a lane.
constexpr int kMaxVectorWidth = 32 * 2 * 256;

bool fits_registers(int64_t hidden) { return hidden % 8 == 0 && hidden <= kMaxVectorWidth; }

template <typename T>
const void *norm_kernel(int nv, bool staged)
{
    return nv == 1 ? (staged ? reinterpret_cast<void *>(&taco_norm_kernel<T, 1, true>)
                             : reinterpret_cast<void *>(&taco_norm_kernel<T, 1, false>))
                   : (staged ? reinterpret_cast<void *>(&taco_norm_kernel<T, 2, true>)
                             : reinterpret_cast<void *>(&taco_norm_kernel<T, 2, false>));
}

template <typename T>
cudaError_t norm_vectors(const NormArgs &a, int sms, cudaStream_t stream)
{
    NormArgs args = a;
    const int nv = a.hidden <= 256 ? 1 : 2;
    int warps = static_cast<int>((a.hidden + 256 * nv - 1) / (256 * nv));
    // As many row groups as fit the CTA, but no more than spread the rows over all SMs; at most 15 barriers.
    const int64_t fit = std::min(kNormThreads / 32 / warps, warps == 1 ? 32 : 15), spread = (a.rows + sms - 1) / sms;
    int groups = static_cast<int>(std::min(fit, spread));
    const int64_t ctas = (a.rows + groups - 1) / groups;
    const bool staged = ctas > sms && (a.weight || a.bias);
    void *p[] = {&args, &warps, &groups};
    return launch_kernel(norm_kernel<T>(nv, staged), static_cast<int>(std::min<int64_t>(ctas, sms)), warps * groups * 32,
                         staged ? 8 * static_cast<size_t>(a.hidden) : 0, stream, p);
}

template <typename T>
cudaError_t norm_any(const NormArgs &a, int sms, cudaStream_t stream)
{
    if (fits_registers(a.hidden))
        return norm_vectors<T>(a, sms, stream);
    NormArgs args = a;
    void *p[] = {&args};
    return launch_kernel(reinterpret_cast<void *>(&taco_norm_any_kernel<T>), row_grid(a.rows, sms, 8), kRowThreads, 0,
                         stream, p);
}

template <typename T>
const void *norm_grad_kernel(int nv, bool records)
{
    return nv == 1   ? (records ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 1, true>)
                                : reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 1, false>))
           : nv == 2 ? (records ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 2, true>)
                                : reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 2, false>))
                     : (records ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 4, true>)
                                : reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 4, false>));
}

constexpr size_t kMaxShared = 225 * 1024;

template <typename T>
cudaError_t norm_grad_any(NormGradArgs *a, int sms, cudaStream_t stream)
{
    const int64_t C = a->hidden;
    if (fits_registers(C)) {
        const int nv = C <= 256 ? 1 : C <= kGradThreads / 32 * 512 ? 2 : 4;
        int warps = static_cast<int>((C + 256 * nv - 1) / (256 * nv));
        const int64_t fit = std::min(kGradThreads / 32 / warps, 15), spread = (a->rows + sms - 1) / sms;
        int groups = static_cast<int>(std::min(fit, spread));
        const int threads = warps * groups * 32;
        const size_t weight = a->weight ? static_cast<size_t>(C * 4 + 15) / 16 * 16 : 0;
        const size_t stage = static_cast<size_t>(1 + (a->x != nullptr) + (a->dsummed != nullptr)) * nv * threads * 8 * sizeof(T);
        int stages = 4;
        while (stages > 1 && weight + stages * stage > kMaxShared)
            stages--;
        const size_t smem = weight + std::max<size_t>(stages * stage, groups > 1 ? 8 * static_cast<size_t>(C) : 0);
        if (smem <= kMaxShared) {
            a->nparts = static_cast<int>(std::min({(a->rows + groups - 1) / groups, static_cast<int64_t>(sms),
                                                   static_cast<int64_t>(kMaxColumnParts)}));
            void *p[] = {a, &warps, &groups, &stages};
            return launch_kernel(norm_grad_kernel<T>(nv, !a->x), a->nparts, threads, smem, stream, p);
        }
    }
    void *p[] = {a};
    cudaError_t e = launch_kernel(reinterpret_cast<void *>(&taco_norm_grad_any_kernel<T>), row_grid(a->rows, sms, 8),
                                  kRowThreads, 0, stream, p);
    if (e == cudaSuccess && a->parts)
        e = launch_kernel_2d(reinterpret_cast<void *>(&taco_norm_grad_columns_kernel<T>),
                             static_cast<unsigned>((a->hidden + 127) / 128), static_cast<unsigned>(a->nparts), 128, 0, stream, p);
    return e;
}

template <typename T>
cudaError_t init_norm_type()
{
    cudaError_t e = cudaSuccess;
    for (int nv = 1; nv <= 2 && e == cudaSuccess; nv++)
        e = cudaFuncSetAttribute(norm_kernel<T>(nv, true), cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * kMaxVectorWidth);
    for (int i = 0; i < 6 && e == cudaSuccess; i++)
        e = cudaFuncSetAttribute(norm_grad_kernel<T>(1 << i / 2, i % 2 != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kMaxShared));
    return e;
}

}  // namespace

cudaError_t launch_column_sums(const float *parts, int nparts, int64_t n, void *out, void *out2, int dtype,
                               cudaStream_t stream)
{
    void *p[] = {&parts, &nparts, &n, &out, &out2, &dtype};
    return launch_kernel_2d(reinterpret_cast<void *>(&taco_column_sums_kernel), static_cast<unsigned>((n + 31) / 32),
                            out2 ? 2u : 1u, 1024, 0, stream, p);
}

cudaError_t init_norm()
{
    cudaError_t e = init_norm_type<__nv_bfloat16>();
    if (e == cudaSuccess)
        e = init_norm_type<__half>();
    return e == cudaSuccess ? init_norm_type<float>() : e;
}

cudaError_t launch_norm(int dtype, const NormArgs &a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? norm_any<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? norm_any<__half>(a, sms, stream)
                               : norm_any<float>(a, sms, stream);
}

cudaError_t launch_norm_grad(int dtype, NormGradArgs *a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? norm_grad_any<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? norm_grad_any<__half>(a, sms, stream)
                               : norm_grad_any<float>(a, sms, stream);
}

}  // namespace taco
