// taco_layernorm_grad.cu -- gradients of the layer norm, from its input or from
// 8-bit checkpoints, and the reduction of the parameters' gradients, for GB300
// (sm_103a).  With a = dy weight:
//   c1 = sum a / C,  c2 = sum a xhat / C,  dx = rstd (a - c1 - xhat c2) [+ dsummed],
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy,
// xhat from (x, mean, rstd) or from records.
#include "taco_norm.cuh"

namespace taco {
namespace {

// ---------------------------------------------------------------------------
// Odd widths too large for shared memory: one CTA per row, element by element
// ---------------------------------------------------------------------------

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
        const float rstd = a.rstd[row], mean = a.mean[row];
        auto xhat = [&](int64_t c) {
            return (to_float(static_cast<const T *>(a.x)[row * C + c]) - mean) * rstd;
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
        const float xh = (to_float(static_cast<const T *>(a.x)[row * C + c]) - a.mean[row]) * a.rstd[row];
        dw = fmaf(g, xh, dw);
        db += g;
    }
    a.parts[static_cast<int64_t>(blockIdx.y) * C + c] = dw;
    a.parts[static_cast<int64_t>(a.nparts + blockIdx.y) * C + c] = db;
}

// ---------------------------------------------------------------------------
// Widths of whole vectors of eight
// ---------------------------------------------------------------------------

// xhat of eight columns from c on.
template <typename T>
__device__ __forceinline__ F8 load_normalised(const NormGradArgs &a, int64_t row, int64_t c, float mean, float rstd)
{
    F8 f;
    if (a.x) {
        f = unpack(load_raw8(static_cast<const T *>(a.x) + row * a.hidden + c));
#pragma unroll
        for (int i = 0; i < 4; i++)
            f.v[i] = mul2(add2(f.v[i], both(-mean)), both(rstd));
    } else {
        const int64_t k = (row * a.hidden + c) / a.block;
        const uint8_t *rec = a.packed + k * (a.block + 8);
        f = codes8_to_float(*reinterpret_cast<const uint2 *>(rec + (row * a.hidden + c - k * a.block)), a.code);
        const float s = record_s(rec, a.block);
#pragma unroll
        for (int i = 0; i < 4; i++)
            f.v[i] = mul2(f.v[i], both(s));
    }
    return f;
}

// Rows too wide for registers and shared memory: dx with a CTA a row, read twice,
// and the column sums in a pass of their own.
constexpr int kWideThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kWideThreads) taco_norm_grad_wide_kernel(NormGradArgs a)
{
    __shared__ float part[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row], mean = a.x ? a.mean[row] : 0.f;
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
        float2 t1 = both(0.f), t2 = both(0.f);
        for (int64_t c = threadIdx.x * 8; c < C; c += kWideThreads * 8) {
            const F8 w = weighted(c), xh = load_normalised<T>(a, row, c, mean, rstd);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                t1 = add2(t1, w.v[i]);
                t2 = fma2(w.v[i], xh.v[i], t2);
            }
        }
        const float c1 = cta_sum(t1.x + t1.y, part) / static_cast<float>(C), c2 = cta_sum(t2.x + t2.y, part) / static_cast<float>(C);
        for (int64_t c = threadIdx.x * 8; c < C; c += kWideThreads * 8) {
            F8 w = weighted(c);
            const F8 xh = load_normalised<T>(a, row, c, mean, rstd);
#pragma unroll
            for (int i = 0; i < 4; i++)
                w.v[i] = mul2(fma2(xh.v[i], both(-c2), add2(w.v[i], both(-c1))), both(rstd));
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
__global__ void __launch_bounds__(128) taco_norm_grad_wide_columns_kernel(NormGradArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden, c = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) * 8;
    if (c >= C)
        return;
    F8 dw, db;
#pragma unroll
    for (int i = 0; i < 4; i++)
        dw.v[i] = db.v[i] = both(0.f);
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < a.rows; row += a.nparts) {
        const F8 g = unpack(load_raw8(static_cast<const T *>(a.dy) + row * C + c));
        const F8 xh = load_normalised<T>(a, row, c, a.x ? a.mean[row] : 0.f, a.rstd[row]);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            dw.v[i] = fma2(g.v[i], xh.v[i], dw.v[i]);
            db.v[i] = add2(db.v[i], g.v[i]);
        }
    }
    store_raw8(a.parts + static_cast<int64_t>(blockIdx.y) * C + c, pack<float>(dw));
    store_raw8(a.parts + static_cast<int64_t>(a.nparts + blockIdx.y) * C + c, pack<float>(db));
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
// CODE: code format of the records, or -1 to read x.
template <typename T, int NV, int CODE, bool FULL>
__global__ void __launch_bounds__(kGradThreads, 1)
taco_norm_grad_kernel(NormGradArgs a, int warps, int groups, int stages)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // weight, then the copies
    __shared__ float2 sums[2][32];
    grid_launch_dependents();
    constexpr bool RECORDS = CODE >= 0;
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
    uint8_t *ring = dynamic + 4 * C;
    const uint32_t ring_at = smem_addr(ring);
    int col[NV];
#pragma unroll
    for (int j = 0; j < NV; j++)
        col[j] = ((warp * NV + j) * 32 + lane) * 8;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group, step = static_cast<int64_t>(gridDim.x) * groups;
    if (warp == 0 && lane < 2 && first + lane * step < a.rows) {
        // the group's first rows on their way to L2 while the kernel before still runs
        const int64_t at = (first + lane * step) * C;
        bulk_prefetch_l2(static_cast<const T *>(a.dy) + at, C * static_cast<int>(sizeof(T)));
        if (!RECORDS)
            bulk_prefetch_l2(static_cast<const T *>(a.x) + at, C * static_cast<int>(sizeof(T)));
        if (a.dsummed)
            bulk_prefetch_l2(static_cast<const T *>(a.dsummed) + at, C * static_cast<int>(sizeof(T)));
    }
    grid_dependency_wait();
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            uint32_t to = ring_at + static_cast<uint32_t>(stage * stage_bytes) + threadIdx.x * 16u;
            auto piece = [&](const void *src) {
#pragma unroll
                for (int j = 0; j < NV; j++)
#pragma unroll
                    for (int k = 0; k < kUnits; k++, to += unit)
                        if (FULL || col[j] < C)
                            copy16<T>(to, reinterpret_cast<const uint4 *>(static_cast<const T *>(src) + row * C + col[j]) + k);
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
            next_rstd = a.rstd[row];
            if (!RECORDS)
                next_mean = a.mean[row];
        }
    };
    for (int i = 0; i < stages - 1; i++)
        copy_row(first + i * step, i);
    fetch(first);
    for (int c = threadIdx.x * 8; c < C; c += blockDim.x * 8)
        stage_param8(sweight, a.weight, a.param_dtype, c, C);
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
        // q and f with xhat = q f (f one factor a vector; 1 where xhat comes from x).
        float factor[NV];
        if (RECORDS) {
#pragma unroll
            for (int j = 0; j < NV; j++)
                if (FULL || col[j] < C)
                    factor[j] = record_s(rec + (col[j] >> shift) * (a.block + 8), a.block);
        }
        auto normalised = [&](int j) {
            if (RECORDS)
                return codes8_to_float(*reinterpret_cast<const uint2 *>(rec + col[j] + (col[j] >> shift) * 8), CODE);
            F8 f = vector(1, j);
#pragma unroll
            for (int i = 0; i < 4; i++)
                f.v[i] = mul2(add2(f.v[i], both(-mean)), both(rstd));
            return f;
        };
        auto weighted = [&](int j, const F8 &g) {
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
                const F8 w = weighted(j, vector(0, j)), q = normalised(j);
                float2 t = RECORDS ? both(0.f) : t2;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    t1 = add2(t1, w.v[i]);
                    t = fma2(w.v[i], q.v[i], t);
                }
                t2 = RECORDS ? fma2(t, both(factor[j]), t2) : t;
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
                const F8 g = vector(0, j), q = normalised(j);
                const float f = RECORDS ? factor[j] : 1.f;
                asm volatile("" ::: "memory");   // the weights are read again rather than kept over the row sums
                F8 w = weighted(j, g);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    dw[j].v[i] = fma2(RECORDS ? mul2(g.v[i], both(f)) : g.v[i], q.v[i], dw[j].v[i]);
                    db[j].v[i] = add2(db[j].v[i], g.v[i]);
                    w.v[i] = mul2(fma2(q.v[i], both(-c2 * f), add2(w.v[i], both(-c1))), both(rstd));
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
            next_rstd = a.rstd[row];
            next_mean = a.mean[row];
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

template <typename T>
const void *norm_grad_odd_kernel(int nv)
{
    return nv == 1   ? reinterpret_cast<void *>(&taco_norm_grad_odd_kernel<T, 1>)
           : nv == 2 ? reinterpret_cast<void *>(&taco_norm_grad_odd_kernel<T, 2>)
                     : reinterpret_cast<void *>(&taco_norm_grad_odd_kernel<T, 4>);
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

template <typename T, int CODE>
const void *norm_grad_kernel(int nv, bool full)
{
    return nv == 1   ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 1, CODE, false>)
           : nv == 2 ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 2, CODE, false>)
           : full    ? reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 4, CODE, true>)
                     : reinterpret_cast<void *>(&taco_norm_grad_kernel<T, 4, CODE, false>);
}

// code: -1 to read x.
template <typename T>
const void *norm_grad_kernel(int nv, int code, bool full)
{
    return code < 0    ? norm_grad_kernel<T, -1>(nv, full)
           : code == 0 ? norm_grad_kernel<T, 0>(nv, full)
           : code == 1 ? norm_grad_kernel<T, 1>(nv, full)
                       : norm_grad_kernel<T, 2>(nv, full);
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
        const size_t weight = static_cast<size_t>(4 * C);
        const size_t place = static_cast<size_t>(1 + !records + (a->dsummed != nullptr)) * nv * warps * 256 * sizeof(T) +
                             (records ? (C / a->block * (a->block + 8) + 8 + 15) / 16 * 16 : 0);
        // fewer groups where their rows do not fit, with records three of each
        while (groups > 1 && (weight + groups * place > max_shared<T>(180) || (records && ring_stages(weight, groups * place) < 3)))
            groups--;
        const int threads = warps * groups * 32;
        const size_t stage = groups * place;
        int stages = std::max(ring_stages(weight, stage, max_shared<T>(180)), records ? std::min(ring_stages(weight, stage), 3) : 1);
        const size_t smem = weight + std::max<size_t>(stages * stage, groups > 1 ? 8 * static_cast<size_t>(C) * groups : 0);
        if (smem <= kMaxShared && (!records || stages >= 3)) {
            a->nparts = static_cast<int>(std::min({(a->rows + groups - 1) / groups, static_cast<int64_t>(sms),
                                                   static_cast<int64_t>(kMaxColumnParts)}));
            void *p[] = {a, &warps, &groups, &stages};
            return launch_kernel(norm_grad_kernel<T>(nv, records ? a->code : -1, C == warps * nv * 256), a->nparts, threads, smem, stream, p);
        }
    }
    if (C % 8 == 0) {
        // about eight CTAs of 128 threads an SM
        const int64_t across = (C + 1023) / 1024;
        a->nparts = static_cast<int>(std::min<int64_t>({a->rows, kMaxColumnParts, std::max<int64_t>(1, 8 * sms / across)}));
        void *p[] = {a};
        cudaError_t e = launch_kernel(reinterpret_cast<void *>(&taco_norm_grad_wide_kernel<T>), row_grid(a->rows, sms, 4), kWideThreads, 0,
                                      stream, p);
        if (e == cudaSuccess && a->parts)
            e = launch_kernel_2d(reinterpret_cast<void *>(&taco_norm_grad_wide_columns_kernel<T>), static_cast<unsigned>(across),
                                 static_cast<unsigned>(a->nparts), 128, 0, stream, p);
        return e;
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
cudaError_t init_norm_grad_type()
{
    for (int nv = 1; nv <= 4; nv *= 2)
        for (int i = 0; i < 9; i++) {
            const cudaError_t e = cudaFuncSetAttribute(i < 8 ? norm_grad_kernel<T>(nv, i / 2 - 1, i & 1) : norm_grad_odd_kernel<T>(nv),
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

cudaError_t init_norm_grad()
{
    cudaError_t e = init_norm_grad_type<__nv_bfloat16>();
    if (e == cudaSuccess)
        e = init_norm_grad_type<__half>();
    return e == cudaSuccess ? init_norm_grad_type<float>() : e;
}

cudaError_t launch_norm_grad(int dtype, NormGradArgs *a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? norm_grad_any<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? norm_grad_any<__half>(a, sms, stream)
                               : norm_grad_any<float>(a, sms, stream);
}

}  // namespace taco

