// taco_train.cuh -- device-side building blocks of the training operators
// (layer norm, GELU, weight gradient): typed loads and stores of eight
// consecutive elements, checkpoint records and warp reductions.
//
// A checkpoint record is a DS-only record [codes | alpha = 1 | s] whose scale
// is a power of two: s = 2^e with the least e >= -126 for which c = max|u| of
// the block has c <= Q_max s.  The products q s of all three code formats then
// hold at most eight significant bits, so they are exact in bf16 (above bf16's
// subnormal range) and a tensor-core product with a checkpoint rounds nothing.
// E4M3 and E5M2 keep their relative precision under any scale; INT8 gives up
// at most one of its bits.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "taco_device.cuh"
#include "taco_train.h"

namespace taco {

// Fault flag of the weight gradient, next to those of the codec (taco_device.cuh).
constexpr uint32_t kFaultWeightGrad = 16u;

// ---------------------------------------------------------------------------
// Typed elements
// ---------------------------------------------------------------------------

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Eight consecutive elements as loaded (16 bytes, or 32 for binary32).
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T *p)
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); i++)
        r.v[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}

__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&f)[8])
{
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int i = 0; i < 8; i++)
        f[i] = __uint_as_float(w[i]);
}

__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float (&f)[8])
{
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void unpack8(const Raw8<__half> &r, float (&f)[8])
{
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 v = f16x2_to_float2(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

__device__ __forceinline__ Raw8<float> pack8(const float (&f)[8], const float *)
{
    Raw8<float> r;
    r.v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    r.v[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    return r;
}

__device__ __forceinline__ Raw8<__nv_bfloat16> pack8(const float (&f)[8], const __nv_bfloat16 *)
{
    Raw8<__nv_bfloat16> r;
    r.v[0] = make_uint4(float2_to_bf16x2(f[0], f[1]), float2_to_bf16x2(f[2], f[3]), float2_to_bf16x2(f[4], f[5]),
                        float2_to_bf16x2(f[6], f[7]));
    return r;
}

__device__ __forceinline__ uint32_t float2_to_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ Raw8<__half> pack8(const float (&f)[8], const __half *)
{
    Raw8<__half> r;
    r.v[0] = make_uint4(float2_to_f16x2(f[0], f[1]), float2_to_f16x2(f[2], f[3]), float2_to_f16x2(f[4], f[5]),
                        float2_to_f16x2(f[6], f[7]));
    return r;
}

// Eight values as four pairs, for packed binary32 arithmetic.
struct F8 {
    float2 v[4];
};

template <typename T>
__device__ __forceinline__ F8 unpack(const Raw8<T> &r)
{
    float f[8];
    unpack8(r, f);
    return F8{{make_float2(f[0], f[1]), make_float2(f[2], f[3]), make_float2(f[4], f[5]), make_float2(f[6], f[7])}};
}

template <typename T>
__device__ __forceinline__ Raw8<T> pack(const F8 &x)
{
    const float f[8] = {x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y, x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y};
    return pack8(f, static_cast<const T *>(nullptr));
}

template <typename T>
__device__ __forceinline__ void store_raw8(T *p, const Raw8<T> &r)
{
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); i++)
        reinterpret_cast<uint4 *>(p)[i] = r.v[i];
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight consecutive parameters of run-time type from i on (i a multiple of 8).
__device__ __forceinline__ void load_param8(const void *p, int dtype, int64_t i, float (&f)[8])
{
    if (dtype == kTypeF32)
        unpack8(load_raw8(static_cast<const float *>(p) + i), f);
    else if (dtype == kTypeF16)
        unpack8(load_raw8(static_cast<const __half *>(p) + i), f);
    else
        unpack8(load_raw8(static_cast<const __nv_bfloat16 *>(p) + i), f);
}

__device__ __forceinline__ F8 load_param_f8(const void *p, int dtype, int64_t i)
{
    float f[8];
    load_param8(p, dtype, i, f);
    return F8{{make_float2(f[0], f[1]), make_float2(f[2], f[3]), make_float2(f[4], f[5]), make_float2(f[6], f[7])}};
}

// Value i of a parameter array of run-time type (uniform over the grid).
__device__ __forceinline__ float load_param(const void *p, int dtype, int64_t i)
{
    if (dtype == kTypeF32)
        return static_cast<const float *>(p)[i];
    if (dtype == kTypeF16)
        return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ void store_param(void *p, int dtype, int64_t i, float v)
{
    if (dtype == kTypeF32)
        static_cast<float *>(p)[i] = v;
    else if (dtype == kTypeF16)
        static_cast<__half *>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------------------
// Records
// ---------------------------------------------------------------------------

// Bits of max over non-negative floats given as |x|'s bit patterns: integer
// order equals float order, and infinities and NaN sort above every finite
// value, so a non-finite element is never lost in the maximum.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The block's scale from its maximum's bits: 2^e as above; 0 for an all-zero
// block; NaN when an element is not finite, so that the block decodes to NaN.
// *inv receives 1 / s (0 for a zero or non-finite block: all codes are zero).
__device__ __forceinline__ float record_scale(uint32_t max_bits, int code, float *inv)
{
    // Q_max = mantissa * 2^shift: 1.75 * 2^8, 1.75 * 2^15, 1.984375 * 2^6.  Adding what a mantissa may lack of 2
    // carries into the exponent just where c's mantissa exceeds Q_max's.
    const uint32_t shift = code == 0 ? 8u : code == 1 ? 15u : 6u, room = code == 2 ? 0x1ffffu : 0x1fffffu;
    const int bits = max(static_cast<int>(((max_bits + room) & 0x7f800000u) - (shift << 23)), 0x00800000);
    const bool ordinary = max_bits - 1u < 0x7f7fffffu;
    *inv = ordinary ? __int_as_float(0x7f000000 - bits) : 0.f;
    return ordinary ? __int_as_float(bits) : max_bits == 0u ? 0.f : __uint_as_float(0x7fc00000u);
}

// Eight code bytes as floats.
__device__ __forceinline__ F8 codes8_to_float(uint2 c, int code)
{
    F8 f;
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float2 a, b;
        if (code == 2) {
            int8x4_to_float(w[h], a, b);
        } else if (code == 0) {
            a = e4m3x2_to_float2(w[h] & 0xffffu);
            b = e4m3x2_to_float2(w[h] >> 16);
        } else {
            a = e5m2x2_to_float2(w[h] & 0xffffu);
            b = e5m2x2_to_float2(w[h] >> 16);
        }
        f.v[2 * h] = a;
        f.v[2 * h + 1] = b;
    }
    return f;
}

// A record's s.  Checkpoints are DS-only records, whose alpha is 1: it is not read.
__device__ __forceinline__ float record_s(const uint8_t *rec, int block)
{
    return *reinterpret_cast<const float *>(rec + block + 4);
}

// The scale of the block that this lane's eight values belong to and their
// codes.  A warp's vector holds 256 consecutive elements, lane l those from 8 l
// on, so a block of B <= 256 lies in B / 8 neighbouring lanes; a block of 512 is
// the two vectors of a pair, whose maxima the caller joins.
__device__ __forceinline__ uint32_t block_max(const F8 &u, int block)
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++)
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(u.v[i].x)), "f"(fabsf(u.v[i].y)));
    uint32_t top = abs_bits(m);                            // a NaN's bits are above infinity's
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
        if (8 * d < block)
            top = max(top, __shfl_xor_sync(kFullMask, top, d));
    return top;
}

// Writes this lane's codes to `at` and, from the lane that holds the block's
// last ones, (1, s) behind them.  `from`: first element's place in the block.
template <int CODE>
__device__ __forceinline__ void write_codes(const F8 &u, uint32_t top, uint8_t *at, int from, int block)
{
    float inv;
    const float s = record_scale(top, CODE, &inv);
    const uint2 q = make_uint2(encode4_scaled(CODE, u.v[0], u.v[1], inv), encode4_scaled(CODE, u.v[2], u.v[3], inv));
    *reinterpret_cast<uint2 *>(at) = inv == 0.f ? make_uint2(0u, 0u) : q;
    if (from + 8 == block)
        *reinterpret_cast<float2 *>(at + 8) = make_float2(1.f, s);
}

// Records of NV vectors of eight a lane, vector j starting at column col[j] of a
// row of C; `row` is the row's first record byte.
template <int NV, int CODE>
__device__ __forceinline__ void write_records(const F8 (&u)[NV], const int (&col)[NV], int C, uint8_t *row, int block)
{
    uint32_t top[NV];
#pragma unroll
    for (int j = 0; j < NV; j++)
        top[j] = block_max(u[j], block);
    if (NV > 1 && block == 512) {
#pragma unroll
        for (int j = 0; j + 1 < NV; j += 2)
            top[j] = top[j + 1] = max(top[j], top[j + 1]);
    }
    const int shift = 31 - __clz(block);
#pragma unroll
    for (int j = 0; j < NV; j++)
        if (col[j] < C)
            write_codes<CODE>(u[j], top[j], row + col[j] + (col[j] >> shift) * 8, col[j] & (block - 1), block);
}

// ---------------------------------------------------------------------------
// Reductions
// ---------------------------------------------------------------------------

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFullMask, v, d);
    return v;
}

// Sum of v over the CTA (whole warps), the same for every thread; `part` holds
// 32 floats and is free again after the call.
__device__ __forceinline__ float cta_sum(float v, float *part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0)
        part[warp] = v;
    __syncthreads();
    v = warp_sum(lane < warps ? part[lane] : 0.f);
    __syncthreads();
    return v;
}

}  // namespace taco
