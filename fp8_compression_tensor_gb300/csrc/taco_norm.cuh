// taco_norm.cuh -- what the layer norm's forward and backward kernels share:
// the layout of a row over a group of warps, asynchronous copies of rows, and
// the host's choice of shapes.
#pragma once

#include <algorithm>

#include "taco_kernels.h"
#include "taco_train.cuh"

namespace taco {
namespace {

constexpr int kRowThreads = 256;


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
// A lane's eight binary32 values are two copies of 16 bytes, each of half a
// 32-byte sector, so these go through L1 (.ca) and the second one finds the
// sector there: 8192 x 4096 with a residual takes 84 us forward and 94 backward,
// past L1 it took 123 and 142.  Rows of 16-bit elements pass it by (.cg): through
// it, 26 -> 33 us.
template <typename T>
__device__ __forceinline__ void copy16(uint32_t to, const void *from)
{
    if (sizeof(T) == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// A copy of whole lines by consecutive lanes, reading `bytes` of the 16 and writing zeros for the others.
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
    float f[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (from)
        load_param8(from, dtype, c, f);
    *reinterpret_cast<float4 *>(p + c / 2) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(p + C / 2 + c / 2) = make_float4(f[4], f[5], f[6], f[7]);
}

// Widths that are no multiple of 8: the same layout with a lane's eight elements 32 apart, so a
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

// Shared memory for the rows of a type.  Binary32 rows are copied through L1,
// which has what shared memory leaves of 256 KB: with about 60 KB (forward) and
// 76 KB (backward) of it the copies' second halves are still there.  8192 x 4096
// with a residual takes 84 us forward, 104 at 228 KB of shared memory; backward 94
// against 120 at 213 KB.
template <typename T>
constexpr size_t max_shared(int kb)
{
    return sizeof(T) == 4 ? static_cast<size_t>(kb) * 1024 : kMaxShared;
}

// Rows in flight: up to four in the shared memory that the parameters leave.
int ring_stages(size_t params, size_t stage, size_t limit = kMaxShared)
{
    int stages = 4;
    while (stages > 1 && params + stages * stage > limit)
        stages--;
    return stages;
}

}  // namespace
}  // namespace taco
