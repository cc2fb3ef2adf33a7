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

// Sum over the 16 lanes of a half warp.
__device__ __forceinline__ float half_warp_sum(float v)
{
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFullMask, v, d);
    return v;
}

// 1 / sqrt(v): the hardware's estimate and one Newton step.
__device__ __forceinline__ float inv_sqrt(float v)
{
    const float r = rsqrtf(v);
    return v > 0.f && v < 3.0e38f ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
}

constexpr int kNormThreads = 768, kGradThreads = 512;   // the backward pass keeps 64 column sums a thread

// Rows come to shared memory `stages` rows ahead by cp.async, 16 bytes at a
// time.  Each thread copies exactly the pieces of x, dy and the like that it
// will read itself, so these need no barrier, only the thread's own wait.
__device__ __forceinline__ void copy16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// The same, reading `bytes` of the 16 and writing zeros for the others.
__device__ __forceinline__ void copy16_part(uint32_t to, const void *from, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the newest `ahead` rows' copies of this thread have landed.
__device__ __forceinline__ void copies_landed(int ahead)
{
    if (ahead == 3)
        asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (ahead == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (ahead == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Parameters in shared memory: of every eight the first four in one plane of
// C / 2 floats and the others in the next, so that a warp's 16-byte reads are
// consecutive (read 32 bytes apart, they would take the banks twice).
__device__ __forceinline__ F8 load_plane8(const float *p, int c, int C)
{
    return unpack(Raw8<float>{{*reinterpret_cast<const uint4 *>(p + c / 2), *reinterpret_cast<const uint4 *>(p + C / 2 + c / 2)}});
}

__device__ __forceinline__ void stage_param8(float *p, const void *from, int dtype, int c, int C)
{
    float f[8];
    load_param8(from, dtype, c, f);
    *reinterpret_cast<float4 *>(p + c / 2) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(p + C / 2 + c / 2) = make_float4(f[4], f[5], f[6], f[7]);
}

// A row's columns over a group of `warps` warps: vector j (of NV) of warp w
// starts at column 256 (w NV + j), lane l holds eight columns from 8 l on.  The
// CTA's groups work on rows of their own.  Many columns a thread keep the two
// row sums cheap: 32 a thread run 8192 x 4096 bf16 with a residual in 47 us, eight a thread
// (twice the warps, two rows a pass) in 58 us.
//
// Statistics with one barrier: each warp sums its values and then their squared
// distances from its own mean p_w = S_w / n_w; with the row's mean m the sum of
// squares is sum_w M_w + n_w (p_w - m)^2.  `sums` alternates between two sets, so
// a set is written again only behind the next row's barrier.
//
// weight and bias stay in shared memory (STAGED) where a CTA has several rows
// to read them for.
// FULL: every lane's every vector lies inside the row, so nothing branches
// between the loads.
template <typename T, int NV, bool STAGED, bool FULL>
__global__ void __launch_bounds__(kNormThreads, 1) taco_norm_kernel(NormArgs a, int warps, int groups, int stages)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // weight, bias (STAGED), then the copies
    __shared__ float2 sums[2][32];
    grid_launch_dependents();
    constexpr int kUnits = sizeof(T) / 2;                 // 16-byte units of eight elements
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int C = static_cast<int>(a.hidden), unit = blockDim.x * 16;
    const float fc = static_cast<float>(C);
    float *sparam = reinterpret_cast<float *>(dynamic);
    const uint8_t *ring = dynamic + (STAGED ? 8 * C : 0) + threadIdx.x * 16;
    const uint32_t ring_at = smem_addr(ring);
    const int row_units = (a.residual ? 2 : 1) * NV * kUnits;
    const int warp_n = min(max(C - warp * 256 * NV, 0), 256 * NV), lane_n = min(max(C - (lane & 15) * 256 * NV, 0), 256 * NV);
    const float warp_inv = warp_n > 0 ? 1.f / static_cast<float>(warp_n) : 0.f;
    const float lane_inv = lane_n > 0 ? 1.f / static_cast<float>(lane_n) : 0.f;   // of warp lane % 16
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    int col[NV];
#pragma unroll
    for (int j = 0; j < NV; j++)
        col[j] = ((warp * NV + j) * 32 + lane) * 8;
    grid_dependency_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group, step = static_cast<int64_t>(gridDim.x) * groups;
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            uint32_t to = ring_at + static_cast<uint32_t>(stage * row_units * unit);
            auto piece = [&](const T *src) {
#pragma unroll
                for (int j = 0; j < NV; j++)
#pragma unroll
                    for (int k = 0; k < kUnits; k++, to += unit)
                        if (FULL || col[j] < C)
                            copy16(to, reinterpret_cast<const uint4 *>(src + row * C + col[j]) + k);
            };
            piece(x);
            if (res)
                piece(res);
        }
        copies_issued();
    };
    for (int i = 0; i < stages - 1; i++)
        copy_row(first + i * step, i);
    if (STAGED) {
        for (int c = threadIdx.x * 8; c < C; c += blockDim.x * 8) {
            if (a.weight)
                stage_param8(sparam, a.weight, a.param_dtype, c, C);
            if (a.bias)
                stage_param8(sparam + C, a.bias, a.param_dtype, c, C);
        }
        __syncthreads();
    }
    auto param = [&](const void *p, int offset, int c) {
        if (STAGED)
            return load_plane8(sparam + offset, c, C);
        return load_param_f8(p, a.param_dtype, c);
    };
    int stage = 0, fill = stages - 1;
    uint32_t side = 0;
    for (int64_t row = first; row < a.rows; row += step, side ^= 1u) {
        copy_row(row + (stages - 1) * step, fill);
        fill = fill + 1 == stages ? 0 : fill + 1;
        copies_landed(stages - 1);
        const uint8_t *mine = ring + static_cast<size_t>(stage) * row_units * unit;
        stage = stage + 1 == stages ? 0 : stage + 1;
        F8 h[NV];
        float2 total = both(0.f);
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
                Raw8<T> v;
#pragma unroll
                for (int k = 0; k < kUnits; k++)
                    v.v[k] = *reinterpret_cast<const uint4 *>(mine + (j * kUnits + k) * unit);
                h[j] = unpack(v);
                if (res) {
#pragma unroll
                    for (int k = 0; k < kUnits; k++)
                        v.v[k] = *reinterpret_cast<const uint4 *>(mine + ((NV + j) * kUnits + k) * unit);
                    const F8 r = unpack(v);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        h[j].v[i] = add2(h[j].v[i], r.v[i]);
                    v = pack<T>(h[j]);
                    store_raw8(static_cast<T *>(a.summed) + row * C + col[j], v);
                    h[j] = unpack(v);
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
                    total = add2(total, h[j].v[i]);
            }
        float sum = warp_sum(total.x + total.y);
        const float pivot = sum * warp_inv;
        float2 squares = both(0.f);
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 d = add2(h[j].v[i], both(-pivot));
                    squares = fma2(d, d, squares);
                }
            }
        float sq = warp_sum(squares.x + squares.y), mean;
        if (warps > 1) {
            float2 *mine_sums = sums[side] + group * warps;
            if (lane == 0)
                mine_sums[warp] = make_float2(sum, sq);
            group_barrier(1 + group, warps * 32);
            // at most 16 warps: the two halves of the warp add the same 16 values
            const int w = lane & 15;
            const float2 v = w < warps ? mine_sums[w] : make_float2(0.f, 0.f);
            mean = half_warp_sum(v.x) / fc;
            const float d = v.x * lane_inv - mean;
            sq = half_warp_sum(fmaf(static_cast<float>(lane_n) * d, d, v.y));
        } else {
            mean = sum / fc;
            const float d = pivot - mean;
            sq = fmaf(fc * d, d, sq);
        }
        const float rstd = inv_sqrt(sq / fc + a.eps);
        if (warp == 0 && lane == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
                F8 y;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    y.v[i] = h[j].v[i] = mul2(add2(h[j].v[i], both(-mean)), both(rstd));
                if (a.weight) {
                    const F8 w = param(a.weight, 0, col[j]);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        y.v[i] = mul2(y.v[i], w.v[i]);
                }
                if (a.bias) {
                    const F8 b = param(a.bias, C, col[j]);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        y.v[i] = add2(y.v[i], b.v[i]);
                }
                store_raw8(static_cast<T *>(a.y) + row * C + col[j], pack<T>(y));
            }
        if (a.packed)
            write_records<NV>(h, col, C, a.packed + row * (C / a.block) * (a.block + 8), a.block, a.code);
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

// The forward pass's layout, so a thread keeps its columns and adds up their
// dweight and dbias in registers over all rows that its group takes.  The
// pieces of a row are read from shared memory twice, for the row's two sums and
// for dx, rather than held in registers next to these sums.
//
// Record bytes (RECORDS) are copied by the whole group, 16 at a time from the
// 16-byte boundary below the row's first one, so they are read behind a barrier:
// the one of the row sums of the row before, ahead of which each thread waits
// for its part of the next row.  A row's place is filled again behind the
// barrier of the row after it, when every thread has left it.
template <typename T, int NV, bool RECORDS, bool FULL>
__global__ void __launch_bounds__(kGradThreads, 1)
taco_norm_grad_kernel(NormGradArgs a, int warps, int groups, int stages)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // weight, then the copies
    __shared__ float2 sums[2][32];
    grid_launch_dependents();
    constexpr int kUnits = sizeof(T) / 2;
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int C = static_cast<int>(a.hidden), unit = blockDim.x * 16;
    const int row_units = (1 + !RECORDS + (a.dsummed != nullptr)) * NV * kUnits;
    const int shift = RECORDS ? 31 - __clz(a.block) : 0;
    const int64_t pitch = RECORDS ? static_cast<int64_t>(C >> shift) * (a.block + 8) : 0;
    const int record_room = RECORDS ? static_cast<int>(pitch + 8 + 15) / 16 * 16 : 0;     // of one group's row
    const int stage_bytes = row_units * unit + groups * record_room;
    const float inv_c = 1.f / static_cast<float>(C);
    float *sweight = reinterpret_cast<float *>(dynamic);
    uint8_t *ring = dynamic + (a.weight ? 4 * C : 0);
    const uint32_t ring_at = smem_addr(ring);
    int col[NV];
#pragma unroll
    for (int j = 0; j < NV; j++)
        col[j] = ((warp * NV + j) * 32 + lane) * 8;
    grid_dependency_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group, step = static_cast<int64_t>(gridDim.x) * groups;
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            uint32_t to = ring_at + static_cast<uint32_t>(stage * stage_bytes) + threadIdx.x * 16u;
            auto piece = [&](const void *src) {
#pragma unroll
                for (int j = 0; j < NV; j++)
#pragma unroll
                    for (int k = 0; k < kUnits; k++, to += unit)
                        if (FULL || col[j] < C)
                            copy16(to, reinterpret_cast<const uint4 *>(static_cast<const T *>(src) + row * C + col[j]) + k);
            };
            piece(a.dy);
            if (!RECORDS)
                piece(a.x);
            if (a.dsummed)
                piece(a.dsummed);
            if (RECORDS) {
                const int64_t at = row * pitch & ~int64_t{15}, left = a.rows * pitch - at;
                const int bytes = static_cast<int>((row + 1) * pitch - at);
                const uint32_t room = ring_at + static_cast<uint32_t>(stage * stage_bytes + row_units * unit + group * record_room);
                for (int c = (warp * 32 + lane) * 16; c < bytes; c += warps * 512)
                    copy16_part(room + c, a.packed + at + c, left - c < 16 ? 8 : 16);
            }
        }
        copies_issued();
    };
    float next_rstd = 0.f, next_mean = 0.f;
    auto fetch = [&](int64_t row) {
        if (row < a.rows) {
            next_rstd = __ldg(a.rstd + row);
            if (!RECORDS)
                next_mean = __ldg(a.mean + row);
        }
    };
    for (int i = 0; i < stages - 1; i++)
        copy_row(first + i * step, i);
    fetch(first);
    if (a.weight) {
        for (int c = threadIdx.x * 8; c < C; c += blockDim.x * 8)
            stage_param8(sweight, a.weight, a.param_dtype, c, C);
    }
    if (RECORDS)
        copies_landed(stages - 2);
    __syncthreads();
    F8 dw[NV], db[NV];
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            dw[j].v[i] = db[j].v[i] = both(0.f);
    int stage = 0, fill = stages - 1;
    uint32_t side = 0;
    for (int64_t row = first; row < a.rows; row += step, side ^= 1u) {
        if (!RECORDS) {
            copy_row(row + (stages - 1) * step, fill);
            copies_landed(stages - 1);
        }
        const uint8_t *mine = ring + static_cast<size_t>(stage) * stage_bytes + threadIdx.x * 16;
        const uint8_t *rec = ring + static_cast<size_t>(stage) * stage_bytes + row_units * unit + group * record_room +
                             (RECORDS ? row * pitch & 15 : 0);
        stage = stage + 1 == stages ? 0 : stage + 1;
        const float rstd = next_rstd, mean = next_mean;
        fetch(row + step);
        // Vector j of the row's piece `tensor`; xhat and dy weight of vector j.
        auto vector = [&](int tensor, int j) {
            Raw8<T> v;
#pragma unroll
            for (int k = 0; k < kUnits; k++)
                v.v[k] = *reinterpret_cast<const uint4 *>(mine + ((tensor * NV + j) * kUnits + k) * unit);
            return unpack(v);
        };
        auto normalised = [&](int j) {
            F8 f;
            if (RECORDS) {
                const uint8_t *block = rec + (col[j] >> shift) * (a.block + 8);
                f = codes8_to_float(*reinterpret_cast<const uint2 *>(block + (col[j] & (a.block - 1))), a.code);
                const float s = meta_factor(*reinterpret_cast<const uint2 *>(block + a.block));
#pragma unroll
                for (int i = 0; i < 4; i++)
                    f.v[i] = mul2(f.v[i], both(s));
            } else {
                f = vector(1, j);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    f.v[i] = mul2(add2(f.v[i], both(-mean)), both(rstd));
            }
            return f;
        };
        auto weighted = [&](int j, const F8 &g) {
            if (!a.weight)
                return g;
            F8 f = load_plane8(sweight, col[j], C);
#pragma unroll
            for (int i = 0; i < 4; i++)
                f.v[i] = mul2(f.v[i], g.v[i]);
            return f;
        };
        float2 t1 = both(0.f), t2 = both(0.f);
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
                const F8 w = weighted(j, vector(0, j)), xh = normalised(j);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    t1 = add2(t1, w.v[i]);
                    t2 = fma2(w.v[i], xh.v[i], t2);
                }
            }
        float s1 = t1.x + t1.y, s2 = t2.x + t2.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            s1 += __shfl_xor_sync(kFullMask, s1, d);
            s2 += __shfl_xor_sync(kFullMask, s2, d);
        }
        if (RECORDS)
            copies_landed(stages - 3);
        if (warps > 1) {
            float2 *mine_sums = sums[side] + group * warps;
            if (lane == 0)
                mine_sums[warp] = make_float2(s1, s2);
            group_barrier(1 + group, warps * 32);
            const int w = lane & 15;
            const float2 v = w < warps ? mine_sums[w] : make_float2(0.f, 0.f);
            s1 = v.x;
            s2 = v.y;
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) {
                s1 += __shfl_xor_sync(kFullMask, s1, d);
                s2 += __shfl_xor_sync(kFullMask, s2, d);
            }
        } else if (RECORDS) {
            __syncwarp();
        }
        if (RECORDS)
            copy_row(row + (stages - 1) * step, fill);
        fill = fill + 1 == stages ? 0 : fill + 1;
        const float c1 = s1 * inv_c, c2 = s2 * inv_c;
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
                const F8 g = vector(0, j), xh = normalised(j);
                F8 w = weighted(j, g);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    dw[j].v[i] = fma2(g.v[i], xh.v[i], dw[j].v[i]);
                    db[j].v[i] = add2(db[j].v[i], g.v[i]);
                    w.v[i] = mul2(fma2(xh.v[i], both(-c2), add2(w.v[i], both(-c1))), both(rstd));
                }
                if (a.dsummed) {
                    const F8 s = vector(RECORDS ? 1 : 2, j);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        w.v[i] = add2(w.v[i], s.v[i]);
                }
                store_raw8(static_cast<T *>(a.dx) + row * C + col[j], pack<T>(w));
            }
    }
    if (!a.parts)
        return;
    // The groups' sums go to the copies' place, [group][dweight, dbias][C] with the layout of load_plane8, and are added in
    // the order of the groups.
    float *acc = reinterpret_cast<float *>(ring) + (groups > 1 ? group * 2 * C : 0);
    copies_landed(0);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; j++)
        if (FULL || col[j] < C) {
            if (groups > 1) {
                const Raw8<float> w = pack<float>(dw[j]), b = pack<float>(db[j]);
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    *reinterpret_cast<uint4 *>(acc + k * (C / 2) + col[j] / 2) = w.v[k];
                    *reinterpret_cast<uint4 *>(acc + C + k * (C / 2) + col[j] / 2) = b.v[k];
                }
            } else {
                store_raw8(a.parts + static_cast<int64_t>(blockIdx.x) * C + col[j], pack<float>(dw[j]));
                store_raw8(a.parts + static_cast<int64_t>(a.nparts + blockIdx.x) * C + col[j], pack<float>(db[j]));
            }
        }
    if (groups == 1)
        return;
    __syncthreads();
    acc = reinterpret_cast<float *>(ring);
    for (int c = threadIdx.x * 4; c < 2 * C; c += blockDim.x * 4) {
        float4 sum = *reinterpret_cast<const float4 *>(acc + c);
        for (int g = 1; g < groups; g++) {
            const float4 v = *reinterpret_cast<const float4 *>(acc + g * 2 * C + c);
            sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
        }
        // place c of the planes: half k of the eight columns from `eight` on
        const int which = c >= C, at = c - which * C, k = at >= C / 2, eight = (at - k * (C / 2)) * 2;
        *reinterpret_cast<float4 *>(a.parts + static_cast<int64_t>(which * a.nparts + blockIdx.x) * C + eight + 4 * k) = sum;
    }
}

// ---------------------------------------------------------------------------
// Widths that are no multiple of 8 (rows that start at any element)
// ---------------------------------------------------------------------------

// The layout of the kernels above, with a lane's eight elements 32 apart, so a
// warp reads and writes consecutive elements.  The group copies its rows to
// shared memory in 16-byte pieces from the boundary below the row's first
// element, and reads them behind a barrier, on the schedule of record bytes
// above.  A row's place holds whole vectors; what lies past the row is ignored.

template <typename T>
__device__ __forceinline__ void copy_odd_row(uint32_t to, const void *base, int64_t row, int64_t rows, int C, int thread, int threads)
{
    const int64_t first = row * C * static_cast<int>(sizeof(T)), at = first & ~int64_t{15}, left = rows * C * static_cast<int>(sizeof(T)) - at;
    const int bytes = static_cast<int>(first - at) + C * static_cast<int>(sizeof(T));
    for (int c = thread * 16; c < bytes; c += threads * 16)
        copy16_part(to + c, static_cast<const uint8_t *>(base) + at + c, left - c < 16 ? static_cast<int>(left - c) : 16);
}

// Where the row's element 0 lies in its place.
template <typename T>
__device__ __forceinline__ int odd_shift(int64_t row, int C)
{
    return static_cast<int>(row * C * static_cast<int>(sizeof(T)) & 15);
}

__host__ __device__ constexpr int odd_room(int width, int element) { return width * element + 32; }

template <typename T, int NV>
__global__ void __launch_bounds__(kNormThreads, 1) taco_norm_odd_kernel(NormArgs a, int warps, int groups, int stages)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // weight, bias, then the copies
    __shared__ float2 sums[2][32];
    grid_launch_dependents();
    constexpr int N = 8 * NV;
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int C = static_cast<int>(a.hidden), c0 = warp * 32 * N + lane;
    const float fc = static_cast<float>(C);
    const int warp_n = min(max(C - warp * 32 * N, 0), 32 * N), lane_n = min(max(C - (lane & 15) * 32 * N, 0), 32 * N);
    const float warp_inv = warp_n > 0 ? 1.f / static_cast<float>(warp_n) : 0.f;
    const float lane_inv = lane_n > 0 ? 1.f / static_cast<float>(lane_n) : 0.f;
    const int room = odd_room(warps * 32 * N, sizeof(T)), tensors = a.residual ? 2 : 1, stage_bytes = groups * tensors * room;
    float *sparam = reinterpret_cast<float *>(dynamic);
    uint8_t *ring = dynamic + (8 * C + 15) / 16 * 16 + group * tensors * room;
    grid_dependency_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group, step = static_cast<int64_t>(gridDim.x) * groups;
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            const uint32_t to = smem_addr(ring) + static_cast<uint32_t>(stage * stage_bytes);
            copy_odd_row<T>(to, a.x, row, a.rows, C, warp * 32 + lane, warps * 32);
            if (a.residual)
                copy_odd_row<T>(to + room, a.residual, row, a.rows, C, warp * 32 + lane, warps * 32);
        }
        copies_issued();
    };
    for (int i = 0; i < stages - 1; i++)
        copy_row(first + i * step, i);
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
        sparam[c] = a.weight ? load_param(a.weight, a.param_dtype, c) : 1.f;
        sparam[C + c] = a.bias ? load_param(a.bias, a.param_dtype, c) : 0.f;
    }
    copies_landed(stages - 2);
    __syncthreads();
    int stage = 0, fill = stages - 1;
    uint32_t side = 0;
    for (int64_t row = first; row < a.rows; row += step, side ^= 1u) {
        const T *x = reinterpret_cast<const T *>(ring + stage * stage_bytes + odd_shift<T>(row, C)) + c0;
        stage = stage + 1 == stages ? 0 : stage + 1;
        float h[N], sum = 0.f, sq = 0.f, mean;
#pragma unroll
        for (int i = 0; i < N; i++)
            h[i] = to_float(x[32 * i]);
        if (a.residual) {
            const T *res = reinterpret_cast<const T *>(reinterpret_cast<const uint8_t *>(x) + room);
            T *out = static_cast<T *>(a.summed) + row * C + c0;
#pragma unroll
            for (int i = 0; i < N; i++) {
                const T v = from_float<T>(h[i] + to_float(res[32 * i]));
                if (c0 + 32 * i < C)
                    out[32 * i] = v;
                h[i] = to_float(v);
            }
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
            h[i] = c0 + 32 * i < C ? h[i] : 0.f;
            sum += h[i];
        }
        sum = warp_sum(sum);
        const float pivot = sum * warp_inv;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float d = c0 + 32 * i < C ? h[i] - pivot : 0.f;
            sq = fmaf(d, d, sq);
        }
        sq = warp_sum(sq);
        copies_landed(stages - 3);
        if (warps > 1) {
            float2 *mine_sums = sums[side] + group * warps;
            if (lane == 0)
                mine_sums[warp] = make_float2(sum, sq);
            group_barrier(1 + group, warps * 32);
            const int w = lane & 15;
            const float2 v = w < warps ? mine_sums[w] : make_float2(0.f, 0.f);
            mean = half_warp_sum(v.x) / fc;
            const float d = v.x * lane_inv - mean;
            sq = half_warp_sum(fmaf(static_cast<float>(lane_n) * d, d, v.y));
        } else {
            __syncwarp();
            mean = sum / fc;
            sq = fmaf(fc * (pivot - mean), pivot - mean, sq);
        }
        copy_row(row + (stages - 1) * step, fill);
        fill = fill + 1 == stages ? 0 : fill + 1;
        const float rstd = inv_sqrt(sq / fc + a.eps);
        if (warp == 0 && lane == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        T *y = static_cast<T *>(a.y) + row * C + c0;
#pragma unroll
        for (int i = 0; i < N; i++)
            if (c0 + 32 * i < C)
                y[32 * i] = from_float<T>(fmaf((h[i] - mean) * rstd, sparam[c0 + 32 * i], sparam[C + c0 + 32 * i]));
    }
}

template <typename T, int NV>
__global__ void __launch_bounds__(kGradThreads, 1) taco_norm_grad_odd_kernel(NormGradArgs a, int warps, int groups, int stages)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // weight, then the copies; then the groups' column sums
    __shared__ float2 sums[2][32];
    grid_launch_dependents();
    constexpr int N = 8 * NV;
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int C = static_cast<int>(a.hidden), c0 = warp * 32 * N + lane;
    const float inv_c = 1.f / static_cast<float>(C);
    const int room = odd_room(warps * 32 * N, sizeof(T)), tensors = a.dsummed ? 3 : 2, stage_bytes = groups * tensors * room;
    float *sweight = reinterpret_cast<float *>(dynamic);                 // whole vectors, zeros past the row
    uint8_t *ring = dynamic + warps * 32 * N * 4 + group * tensors * room;
    grid_dependency_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group, step = static_cast<int64_t>(gridDim.x) * groups;
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            const uint32_t to = smem_addr(ring) + static_cast<uint32_t>(stage * stage_bytes);
            copy_odd_row<T>(to, a.dy, row, a.rows, C, warp * 32 + lane, warps * 32);
            copy_odd_row<T>(to + room, a.x, row, a.rows, C, warp * 32 + lane, warps * 32);
            if (a.dsummed)
                copy_odd_row<T>(to + 2 * room, a.dsummed, row, a.rows, C, warp * 32 + lane, warps * 32);
        }
        copies_issued();
    };
    float next_rstd = 0.f, next_mean = 0.f;
    auto fetch = [&](int64_t row) {
        if (row < a.rows) {
            next_rstd = __ldg(a.rstd + row);
            next_mean = __ldg(a.mean + row);
        }
    };
    for (int i = 0; i < stages - 1; i++)
        copy_row(first + i * step, i);
    fetch(first);
    for (int c = threadIdx.x; c < warps * 32 * N; c += blockDim.x)
        sweight[c] = c >= C ? 0.f : a.weight ? load_param(a.weight, a.param_dtype, c) : 1.f;
    copies_landed(stages - 2);
    __syncthreads();
    const float *weight = sweight + c0;
    float dw[N], db[N];
#pragma unroll
    for (int i = 0; i < N; i++)
        dw[i] = db[i] = 0.f;
    int stage = 0, fill = stages - 1;
    uint32_t side = 0;
    for (int64_t row = first; row < a.rows; row += step, side ^= 1u) {
        const uint8_t *place = ring + stage * stage_bytes + odd_shift<T>(row, C);
        const T *dy = reinterpret_cast<const T *>(place) + c0, *x = reinterpret_cast<const T *>(place + room) + c0,
                *ds = reinterpret_cast<const T *>(place + 2 * room) + c0;
        stage = stage + 1 == stages ? 0 : stage + 1;
        const float rstd = next_rstd, mean = next_mean;
        fetch(row + step);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float w = to_float(dy[32 * i]) * weight[32 * i], xh = (to_float(x[32 * i]) - mean) * rstd;
            s1 += c0 + 32 * i < C ? w : 0.f;
            s2 += c0 + 32 * i < C ? w * xh : 0.f;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            s1 += __shfl_xor_sync(kFullMask, s1, d);
            s2 += __shfl_xor_sync(kFullMask, s2, d);
        }
        copies_landed(stages - 3);
        if (warps > 1) {
            float2 *mine_sums = sums[side] + group * warps;
            if (lane == 0)
                mine_sums[warp] = make_float2(s1, s2);
            group_barrier(1 + group, warps * 32);
            const float2 v = (lane & 15) < warps ? mine_sums[lane & 15] : make_float2(0.f, 0.f);
            s1 = half_warp_sum(v.x);
            s2 = half_warp_sum(v.y);
        } else {
            __syncwarp();
        }
        copy_row(row + (stages - 1) * step, fill);
        fill = fill + 1 == stages ? 0 : fill + 1;
        const float c1 = s1 * inv_c, c2 = s2 * inv_c;
        T *dx = static_cast<T *>(a.dx) + row * C + c0;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float g = to_float(dy[32 * i]), xh = (to_float(x[32 * i]) - mean) * rstd;
            dw[i] = fmaf(g, xh, dw[i]);               // what lies past the row is never written out
            db[i] += g;
            float v = rstd * fmaf(-xh, c2, fmaf(g, weight[32 * i], -c1));
            if (a.dsummed)
                v += to_float(ds[32 * i]);
            if (c0 + 32 * i < C)
                dx[32 * i] = from_float<T>(v);
        }
    }
    if (!a.parts)
        return;
    // The groups' sums, [group][dweight, dbias][C], added in the order of the groups.
    float *shared = reinterpret_cast<float *>(dynamic);
    copies_landed(0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++)
        if (c0 + 32 * i < C) {
            shared[group * 2 * C + c0 + 32 * i] = dw[i];
            shared[group * 2 * C + C + c0 + 32 * i] = db[i];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * C; c += blockDim.x) {
        float sum = shared[c];
        for (int g = 1; g < groups; g++)
            sum += shared[g * 2 * C + c];
        const int which = c >= C;
        a.parts[static_cast<int64_t>(which * a.nparts + blockIdx.x) * C + c - which * C] = sum;
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

// Whole vectors of eight, and at most 16 warps of four vectors a lane.
constexpr int kMaxVectorWidth = 16 * 4 * 256;
constexpr size_t kMaxShared = 225 * 1024;

bool fits_registers(int64_t hidden) { return hidden <= kMaxVectorWidth; }

// Vectors a lane: four, or what a single warp needs for a short row.
int lane_vectors(int64_t hidden) { return hidden <= 256 ? 1 : hidden <= 512 ? 2 : 4; }

// Row groups of a CTA: as many as fit it, but no more than spread the rows over
// all SMs, and one named barrier each (15 besides the CTA's own).
int row_groups(int64_t rows, int warps, int threads, int sms)
{
    const int64_t fit = std::min(threads / 32 / warps, warps == 1 ? 32 : 15), spread = (rows + sms - 1) / sms;
    return static_cast<int>(std::min(fit, spread));
}

template <typename T, bool FLAG>
const void *norm_kernel(int nv, bool full)
{
    return nv == 1   ? reinterpret_cast<void *>(&taco_norm_kernel<T, 1, FLAG, false>)
           : nv == 2 ? reinterpret_cast<void *>(&taco_norm_kernel<T, 2, FLAG, false>)
           : full    ? reinterpret_cast<void *>(&taco_norm_kernel<T, 4, FLAG, true>)
                     : reinterpret_cast<void *>(&taco_norm_kernel<T, 4, FLAG, false>);
}

template <typename T>
const void *norm_kernel(int nv, bool staged, bool full)
{
    return staged ? norm_kernel<T, true>(nv, full) : norm_kernel<T, false>(nv, full);
}

template <typename T>
const void *norm_odd_kernel(int nv)
{
    return nv == 1   ? reinterpret_cast<void *>(&taco_norm_odd_kernel<T, 1>)
           : nv == 2 ? reinterpret_cast<void *>(&taco_norm_odd_kernel<T, 2>)
                     : reinterpret_cast<void *>(&taco_norm_odd_kernel<T, 4>);
}

template <typename T>
const void *norm_grad_odd_kernel(int nv)
{
    return nv == 1   ? reinterpret_cast<void *>(&taco_norm_grad_odd_kernel<T, 1>)
           : nv == 2 ? reinterpret_cast<void *>(&taco_norm_grad_odd_kernel<T, 2>)
                     : reinterpret_cast<void *>(&taco_norm_grad_odd_kernel<T, 4>);
}

// Rows in flight: up to four in the shared memory that the parameters leave.
int ring_stages(size_t params, size_t stage, int most = 4)
{
    while (most > 1 && params + most * stage > kMaxShared)
        most--;
    return most;
}

// Kernel and shape for odd widths; false where three rows do not fit shared memory.
template <typename T>
bool norm_odd(const NormArgs &a, int sms, cudaStream_t stream, cudaError_t *result)
{
    NormArgs args = a;
    const int nv = lane_vectors(a.hidden);
    int warps = static_cast<int>((a.hidden + 256 * nv - 1) / (256 * nv));
    int groups = row_groups(a.rows, warps, kNormThreads, sms);
    const size_t params = (8 * static_cast<size_t>(a.hidden) + 15) / 16 * 16;
    const size_t place = static_cast<size_t>(a.residual ? 2 : 1) * odd_room(warps * nv * 256, sizeof(T));
    while (groups > 1 && ring_stages(params, groups * place) < 3)
        groups--;
    const size_t stage = groups * place;
    int stages = ring_stages(params, stage);
    if (stages < 3)
        return false;
    void *p[] = {&args, &warps, &groups, &stages};
    *result = launch_kernel(norm_odd_kernel<T>(nv), static_cast<int>(std::min<int64_t>((a.rows + groups - 1) / groups, sms)),
                            warps * groups * 32, params + stages * stage, stream, p);
    return true;
}

template <typename T>
bool norm_grad_odd(NormGradArgs *a, int sms, cudaStream_t stream, cudaError_t *result)
{
    const int nv = lane_vectors(a->hidden);
    int warps = static_cast<int>((a->hidden + 256 * nv - 1) / (256 * nv));
    int groups = row_groups(a->rows, warps, kGradThreads, sms);
    const size_t weight = static_cast<size_t>(warps) * nv * 1024;
    const size_t place = static_cast<size_t>(a->dsummed ? 3 : 2) * odd_room(warps * nv * 256, sizeof(T));
    while (groups > 1 && ring_stages(weight, groups * place) < 3)
        groups--;
    const size_t stage = groups * place;
    int stages = ring_stages(weight, stage);
    if (stages < 3)
        return false;
    a->nparts = static_cast<int>(std::min({(a->rows + groups - 1) / groups, static_cast<int64_t>(sms),
                                           static_cast<int64_t>(kMaxColumnParts)}));
    void *p[] = {a, &warps, &groups, &stages};
    *result = launch_kernel(norm_grad_odd_kernel<T>(nv), a->nparts, warps * groups * 32,
                            std::max(weight + stages * stage, 8 * static_cast<size_t>(a->hidden) * groups), stream, p);
    return true;
}

template <typename T>
cudaError_t norm_vectors(const NormArgs &a, int sms, cudaStream_t stream)
{
    NormArgs args = a;
    const int nv = lane_vectors(a.hidden);
    int warps = static_cast<int>((a.hidden + 256 * nv - 1) / (256 * nv));
    int groups = row_groups(a.rows, warps, kNormThreads, sms);
    const int threads = warps * groups * 32;
    const int64_t ctas = (a.rows + groups - 1) / groups;
    const bool staged = ctas > sms && (a.weight || a.bias);
    const size_t params = staged ? 8 * static_cast<size_t>(a.hidden) : 0;
    const size_t stage = static_cast<size_t>(a.residual ? 2 : 1) * nv * threads * 8 * sizeof(T);
    int stages = ring_stages(params, stage);
    void *p[] = {&args, &warps, &groups, &stages};
    return launch_kernel(norm_kernel<T>(nv, staged, a.hidden == warps * nv * 256), static_cast<int>(std::min<int64_t>(ctas, sms)), threads,
                         params + stages * stage, stream, p);
}

template <typename T>
cudaError_t norm_any(const NormArgs &a, int sms, cudaStream_t stream)
{
    cudaError_t result;
    if (fits_registers(a.hidden) && a.hidden % 8 == 0)
        return norm_vectors<T>(a, sms, stream);
    if (fits_registers(a.hidden) && norm_odd<T>(a, sms, stream, &result))
        return result;
    NormArgs args = a;
    void *p[] = {&args};
    return launch_kernel(reinterpret_cast<void *>(&taco_norm_any_kernel<T>), row_grid(a.rows, sms, 8), kRowThreads, 0,
                         stream, p);
}

template <typename T, bool FLAG>
const void *norm_grad_kernel(int nv, bool full)
{
    return nv == 1   ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 1, FLAG, false>)
           : nv == 2 ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 2, FLAG, false>)
           : full    ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 4, FLAG, true>)
                     : reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 4, FLAG, false>);
}

template <typename T>
const void *norm_grad_kernel(int nv, bool records, bool full)
{
    return records ? norm_grad_kernel<T, true>(nv, full) : norm_grad_kernel<T, false>(nv, full);
}

template <typename T>
cudaError_t norm_grad_any(NormGradArgs *a, int sms, cudaStream_t stream)
{
    const int64_t C = a->hidden;
    cudaError_t result;
    if (fits_registers(C) && C % 8 && norm_grad_odd<T>(a, sms, stream, &result))
        return result;
    if (fits_registers(C) && C % 8 == 0) {
        const bool records = !a->x;
        const int nv = lane_vectors(C);
        int warps = static_cast<int>((C + 256 * nv - 1) / (256 * nv));
        int groups = row_groups(a->rows, warps, kGradThreads, sms);
        const int threads = warps * groups * 32;
        const size_t weight = a->weight ? static_cast<size_t>(4 * C) : 0;
        size_t stage = static_cast<size_t>(1 + !records + (a->dsummed != nullptr)) * nv * threads * 8 * sizeof(T);
        if (records)
            stage += static_cast<size_t>(groups) * ((C / a->block * (a->block + 8) + 8 + 15) / 16 * 16);
        int stages = ring_stages(weight, stage);
        const size_t smem = weight + std::max<size_t>(stages * stage, groups > 1 ? 8 * static_cast<size_t>(C) * groups : 0);
        if (smem <= kMaxShared && (!records || stages >= 3)) {
            a->nparts = static_cast<int>(std::min({(a->rows + groups - 1) / groups, static_cast<int64_t>(sms),
                                                   static_cast<int64_t>(kMaxColumnParts)}));
            void *p[] = {a, &warps, &groups, &stages};
            return launch_kernel(norm_grad_kernel<T>(nv, records, C == warps * nv * 256), a->nparts, threads, smem, stream, p);
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
    for (int nv = 1; nv <= 4; nv *= 2)
        for (int i = 0; i < 10; i++) {
            const bool flag = i & 1, full = i & 2;
            const void *kernel = i < 4   ? norm_kernel<T>(nv, flag, full)
                                 : i < 8 ? norm_grad_kernel<T>(nv, flag, full)
                                 : i < 9 ? norm_odd_kernel<T>(nv)
                                         : norm_grad_odd_kernel<T>(nv);
            const cudaError_t e = cudaFuncSetAttribute(kernel,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxShared));
            if (e != cudaSuccess)
                return e;
        }
    return cudaSuccess;
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
