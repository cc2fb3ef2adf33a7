// taco_rms.cuh -- what the RMS norm's forward and backward kernels share.
//
// Rows that start anywhere.  All tensors of a call have one shape and 16-byte
// aligned bases, so a row of any width C is cut into the same whole vectors of
// eight elements in all of them: with shift = row C mod 8 its vector v holds the
// columns 8 v - shift .. 8 v - shift + 7, and only the first and the last reach
// into the neighbouring rows.  A CTA takes rows whose numbers differ by multiples
// of the grid, which is a multiple of 8 (or takes one row a group), so its rows
// have one shift: parameters are staged shifted once, and a thread keeps its
// columns from row to row, which the column sums of a gradient need.  Odd widths
// then cost what their edges do: 8192 x 4097 bf16 with a residual takes 47 us and
// 8192 x 4096 45, where copies to shared memory that are read 32 columns apart (the
// layer norm's way) take 73.
#pragma once

#include "taco_norm.cuh"

namespace taco {
namespace {

// Whether a vector whose first column is c reaches outside the row.
__device__ __forceinline__ bool at_edge(int c, int C) { return c < 0 || c + 8 > C; }

// Zeros for what lies outside the row in `tensors` pieces of a vector whose first column is c, `pitch` bytes apart and
// each in units of 16 bytes `unit` apart (shared memory, this thread's own copies).
template <typename T>
__device__ __forceinline__ void clear_edge(uint8_t *piece, int tensors, int pitch, int unit, int c, int C)
{
    constexpr int kPerUnit = 16 / sizeof(T);
#pragma unroll 1
    for (int t = 0; t < tensors; t++, piece += pitch)
#pragma unroll 1
        for (int i = 0; i < 8; i++)
            if (c + i < 0 || c + i >= C)
                reinterpret_cast<T *>(piece + i / kPerUnit * unit)[i % kPerUnit] = from_float<T>(0.f);
}

// Stores column c on of the row at `row`, element by element inside the row.
template <typename T>
__device__ __forceinline__ void store_edge(T *row, const F8 &f, int c, int C)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (c + 2 * i >= 0 && c + 2 * i < C)
            row[c + 2 * i] = from_float<T>(f.v[i].x);
        if (c + 2 * i + 1 >= 0 && c + 2 * i + 1 < C)
            row[c + 2 * i + 1] = from_float<T>(f.v[i].y);
    }
}

template <typename T, bool ODD>
__device__ __forceinline__ void store_vector(T *row, const F8 &f, int c, int C)
{
    if (ODD && at_edge(c, C))
        store_edge(row, f, c, C);
    else
        store_raw8(row + c, pack<T>(f));
}

// copy16 (taco_norm.cuh) of which `bytes` (0 to 16) are read.
template <typename T>
__device__ __forceinline__ void copy16_upto(uint32_t to, const void *from, int bytes)
{
    if (sizeof(T) == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    else
        copy16_part(to, from, bytes);
}

// Eight parameters from column c on, `fill` outside the row.
__device__ __forceinline__ F8 load_param_edge(const void *p, int dtype, int c, int C, float fill)
{
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        f[i] = c + i >= 0 && c + i < C ? load_param(p, dtype, c + i) : fill;
    return F8{{make_float2(f[0], f[1]), make_float2(f[2], f[3]), make_float2(f[4], f[5]), make_float2(f[6], f[7])}};
}

// Vectors of a row of any shift.
__host__ __device__ constexpr int row_vectors(int64_t hidden) { return static_cast<int>(hidden % 8 ? (hidden + 14) / 8 : hidden / 8); }

// Stages a parameter array in planes of `vectors` vectors, vector v from column 8 v - shift on.
template <bool ODD>
__device__ __forceinline__ void stage_shifted(float *to, const void *from, int dtype, int vectors, int shift, int C, float fill)
{
    for (int v = threadIdx.x; v < vectors; v += blockDim.x) {
        const int c = 8 * v - shift;
        const F8 f = ODD ? load_param_edge(from, dtype, c, C, fill) : load_param_f8(from, dtype, c);
        *reinterpret_cast<float4 *>(to + 4 * v) = make_float4(f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y);
        *reinterpret_cast<float4 *>(to + 4 * (vectors + v)) = make_float4(f.v[2].x, f.v[2].y, f.v[3].x, f.v[3].y);
    }
}

__device__ __forceinline__ F8 load_shifted(const float *p, int v, int vectors)
{
    return unpack(Raw8<float>{{*reinterpret_cast<const uint4 *>(p + 4 * v), *reinterpret_cast<const uint4 *>(p + 4 * (vectors + v))}});
}

// CTAs for `ctas` wanted; for rows that start anywhere a multiple of 8, so that a CTA's rows share their shift, unless
// each CTA has a single row.
inline int shifted_grid(int64_t ctas, int groups, bool odd, int sms)
{
    if (!odd || (groups == 1 && ctas <= sms))
        return static_cast<int>(std::min<int64_t>(ctas, sms));
    return static_cast<int>(std::min<int64_t>((ctas + 7) / 8 * 8, std::max(sms / 8 * 8, 8)));
}

// The sum over a group's warps of v (already summed over the warp), for all of its threads; `sums` is the group's.
__device__ __forceinline__ float group_sum(float v, float *sums, int group, int warp, int warps)
{
    const int lane = threadIdx.x & 31;
    if (warps == 1)
        return v;
    if (lane == 0)
        sums[warp] = v;
    group_barrier(1 + group, warps * 32);
    return warp_sum(lane < warps ? sums[lane] : 0.f);
}

}  // namespace
}  // namespace taco
