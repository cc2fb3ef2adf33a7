// taco_rmsnorm_grad.cu -- gradients of the root-mean-square norm, from its input
// or from 8-bit checkpoints, for GB300 (sm_103a).  With a = dy weight:
//   c = sum a xhat / C,  dx = rstd (a - xhat c) [+ dsummed],
//   dweight = sum over rows of dy xhat,
// xhat = x rstd, or from records.
#include "taco_rms.cuh"

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

// ---------------------------------------------------------------------------
// Rows in shared memory
// ---------------------------------------------------------------------------

// The forward pass's layout, so a thread keeps its columns and adds up their
// dweight in registers over all rows that its group takes.  A row's pieces are
// read from shared memory twice, for the row's sum and for dx, rather than held in
// registers next to these sums.
//
// Record bytes (CODE >= 0) are copied by the whole group, 16 at a time from the
// 16-byte boundary below the row's first one, so they are read behind a barrier:
// the one of the row sum of the row before, ahead of which each thread waits for
// its part of the next row.  A row's place is filled again behind the barrier of
// the row after it, when every thread has left it.
// DIRECT: dsummed does not come to shared memory, where the rows would no longer
// fit, but to L2 a row ahead and is loaded where it is added.  8192 x 11648 bf16 from
// records with dsummed takes 188 us so, and 309 with rows read twice.
// CODE: code format of the records, or -1 to read x.  ODD and FULL as forward.
constexpr int kRmsGradThreads = 512;

template <typename T, int NV, int CODE, bool ODD, bool FULL, bool DIRECT>
__global__ void __launch_bounds__(kRmsGradThreads, 1) taco_rms_grad_kernel(RmsGradArgs a, int warps, int groups, int stages)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // weight, then the copies; then the groups' column sums
    __shared__ float sums[2][32];
    grid_launch_dependents();
    constexpr bool RECORDS = CODE >= 0;
    constexpr int kUnits = sizeof(T) / 2;
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int C = static_cast<int>(a.hidden), unit = blockDim.x * 16, vectors = row_vectors(C);
    const int shift = ODD ? static_cast<int>(blockIdx.x * a.hidden & 7) : 0;
    const int row_units = (1 + !RECORDS + (!DIRECT && a.dsummed)) * NV * kUnits;
    const int block_log = RECORDS ? 31 - __clz(a.block) : 0;
    const int64_t pitch = RECORDS ? static_cast<int64_t>(C >> block_log) * (a.block + 8) : 0;
    const int record_room = RECORDS ? static_cast<int>(pitch + 8 + 15) / 16 * 16 : 0;     // of one group's row
    const int stage_bytes = row_units * unit + groups * record_room;
    const float inv_c = 1.f / static_cast<float>(C);
    float *sweight = reinterpret_cast<float *>(dynamic);
    uint8_t *ring = dynamic + 32 * vectors;
    const uint32_t ring_at = smem_addr(ring);
    const int v0 = warp * NV * 32 + lane;
    int col[NV];
#pragma unroll
    for (int j = 0; j < NV; j++)
        col[j] = (v0 + 32 * j) * 8 - shift;
    bool edges = false;   // whether one of this thread's vectors reaches outside the row
#pragma unroll
    for (int j = 0; j < NV; j++)
        edges = edges || (ODD && col[j] < C && at_edge(col[j], C));
    const int64_t first = ODD ? blockIdx.x + static_cast<int64_t>(gridDim.x) * group : static_cast<int64_t>(blockIdx.x) * groups + group;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    if (warp == 0 && lane < 2 && !ODD && first + lane * step < a.rows) {
        // the group's first rows on their way to L2 while the kernel before still runs
        const int64_t at = (first + lane * step) * C;
        bulk_prefetch_l2(static_cast<const T *>(a.dy) + at, C * static_cast<int>(sizeof(T)));
        if (!RECORDS)
            bulk_prefetch_l2(static_cast<const T *>(a.x) + at, C * static_cast<int>(sizeof(T)));
        if (a.dsummed)
            bulk_prefetch_l2(static_cast<const T *>(a.dsummed) + at, C * static_cast<int>(sizeof(T)));
    }
    grid_dependency_wait();
    const int64_t end = a.rows * a.hidden * static_cast<int>(sizeof(T));   // of the tensors, in bytes
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            // the tensors' last vector may end behind them
            const bool whole = !ODD || (row * C - shift + 8 * vectors) * static_cast<int>(sizeof(T)) <= end;
            uint32_t to = ring_at + static_cast<uint32_t>(stage * stage_bytes) + threadIdx.x * 16u;
            auto piece = [&](const void *tensor) {
                const T *src = static_cast<const T *>(tensor);
#pragma unroll
                for (int j = 0; j < NV; j++)
#pragma unroll
                    for (int k = 0; k < kUnits; k++, to += unit)
                        if (FULL || col[j] < C) {
                            const T *from = src + row * C + col[j] + 8 / kUnits * k;
                            if (!ODD || whole) {
                                copy16<T>(to, from);
                            } else {
                                const int64_t left = end - (row * C + col[j]) * static_cast<int>(sizeof(T)) - 16 * k;
                                copy16_upto<T>(to, left > 0 ? from : src, left >= 16 ? 16 : left > 0 ? static_cast<int>(left) : 0);
                            }
                        }
            };
            piece(a.dy);
            if (!RECORDS)
                piece(a.x);
            if (!DIRECT && a.dsummed)
                piece(a.dsummed);
            if (DIRECT && warp == 0 && lane == 0)
                bulk_prefetch_l2(static_cast<const T *>(a.dsummed) + row * C, C * static_cast<int>(sizeof(T)));
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
    float next_rstd = 0.f;
    auto fetch = [&](int64_t row) {
        if (row < a.rows)
            next_rstd = a.rstd[row];
    };
    for (int i = 0; i < stages - 1; i++)
        copy_row(first + i * step, i);
    fetch(first);
    if (a.weight) {
        stage_shifted<ODD>(sweight, a.weight, a.param_dtype, vectors, shift, C, 0.f);
    } else {
        for (int i = threadIdx.x; i < 8 * vectors; i += blockDim.x)
            sweight[i] = 1.f;
    }
    if (RECORDS)
        copies_landed(stages - 2);
    __syncthreads();
    F8 dw[NV] = {};
    int stage = 0, fill = stages - 1;
    uint32_t side = 0;
    for (int64_t row = first; row < a.rows; row += step, side ^= 1u) {
        if (!RECORDS) {
            copy_row(row + (stages - 1) * step, fill);
            copies_landed(stages - 1);
        }
        uint8_t *mine = ring + static_cast<size_t>(stage) * stage_bytes + threadIdx.x * 16;
        const uint8_t *rec = ring + static_cast<size_t>(stage) * stage_bytes + row_units * unit + group * record_room +
                             (RECORDS ? row * pitch & 15 : 0);
        stage = stage + 1 == stages ? 0 : stage + 1;
        const float rstd = next_rstd;
        fetch(row + step);
        if (ODD && edges) {
#pragma unroll
            for (int j = 0; j < NV; j++)
                if (col[j] < C && at_edge(col[j], C))
                    clear_edge<T>(mine + j * kUnits * unit, 2, NV * kUnits * unit, unit, col[j], C);
        }
        auto vector = [&](int tensor, int j) {
            Raw8<T> v;
#pragma unroll
            for (int k = 0; k < kUnits; k++)
                v.v[k] = *reinterpret_cast<const uint4 *>(mine + ((tensor * NV + j) * kUnits + k) * unit);
            return unpack(v);
        };
        // xhat = q f: codes and their block's scale, or x and rstd
        float factor[NV];
#pragma unroll
        for (int j = 0; j < NV; j++)
            factor[j] = !RECORDS ? rstd : FULL || col[j] < C ? record_s(rec + (col[j] >> block_log) * (a.block + 8), a.block) : 0.f;
        auto unscaled = [&](int j) {
            if (RECORDS)
                return codes8_to_float(*reinterpret_cast<const uint2 *>(rec + col[j] + (col[j] >> block_log) * 8), CODE);
            return vector(1, j);
        };
        float2 total = both(0.f);
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
                F8 w = load_shifted(sweight, v0 + 32 * j, vectors);
                const F8 g = vector(0, j), q = unscaled(j);
                float2 t = both(0.f);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    t = fma2(mul2(w.v[i], g.v[i]), q.v[i], t);
                total = fma2(t, both(factor[j]), total);
            }
        float s = warp_sum(total.x + total.y);
        if (RECORDS)
            copies_landed(stages - 3);
        s = group_sum(s, sums[side] + group * warps, group, warp, warps);
        if (RECORDS) {
            if (warps == 1)
                __syncwarp();
            copy_row(row + (stages - 1) * step, fill);
        }
        fill = fill + 1 == stages ? 0 : fill + 1;
        const float c = s * inv_c;
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
                const F8 g = vector(0, j), q = unscaled(j);
                asm volatile("" ::: "memory");   // the weights are read again rather than kept over the row's sum
                F8 w = load_shifted(sweight, v0 + 32 * j, vectors);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    dw[j].v[i] = fma2(mul2(g.v[i], both(factor[j])), q.v[i], dw[j].v[i]);
                    w.v[i] = mul2(fma2(q.v[i], both(-c * factor[j]), mul2(w.v[i], g.v[i])), both(rstd));
                }
                if (DIRECT || a.dsummed) {
                    const F8 d = DIRECT ? unpack(load_raw8(static_cast<const T *>(a.dsummed) + row * C + col[j])) : vector(RECORDS ? 1 : 2, j);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        w.v[i] = add2(w.v[i], d.v[i]);
                }
                store_vector<T, ODD>(static_cast<T *>(a.dx) + row * C, w, col[j], C);
            }
    }
    if (!a.parts)
        return;
    // The groups' sums go to the copies' place in planes and are added in the order of the groups.
    float *acc = reinterpret_cast<float *>(ring), *out = a.parts + static_cast<int64_t>(blockIdx.x) * C;
    copies_landed(0);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; j++)
        if (FULL || col[j] < C) {
            if (groups > 1) {
                const Raw8<float> w = pack<float>(dw[j]);
                float *to = acc + group * 8 * vectors + 4 * (v0 + 32 * j);
                *reinterpret_cast<uint4 *>(to) = w.v[0];
                *reinterpret_cast<uint4 *>(to + 4 * vectors) = w.v[1];
            } else if (ODD) {
                store_edge(out, dw[j], col[j], C);
            } else {
                store_raw8(out + col[j], pack<float>(dw[j]));
            }
        }
    if (groups == 1)
        return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * vectors; i += blockDim.x) {
        float4 sum = *reinterpret_cast<const float4 *>(acc + 4 * i);
        for (int g = 1; g < groups; g++) {
            const float4 v = *reinterpret_cast<const float4 *>(acc + g * 8 * vectors + 4 * i);
            sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
        }
        // place i of the planes: half k of vector v
        const int k = i >= vectors, v = i - k * vectors, at = 8 * v + 4 * k - shift;
        if (!ODD) {
            *reinterpret_cast<float4 *>(out + at) = sum;
        } else {
            const float f[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (at + e >= 0 && at + e < C)
                    out[at + e] = f[e];
        }
    }
}

template <typename T, int CODE>
const void *rms_grad_kernel(int nv, bool full)
{
    return nv == 1   ? reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 1, CODE, false, false, false>)
           : nv == 2 ? reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 2, CODE, false, false, false>)
           : full    ? reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 4, CODE, false, true, false>)
                     : reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 4, CODE, false, false, false>);
}

// From records with dsummed loaded where it is added (wide rows: four vectors a lane).
template <typename T>
const void *rms_grad_direct_kernel(int code)
{
    return code == 0   ? reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 4, 0, false, false, true>)
           : code == 1 ? reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 4, 1, false, false, true>)
                       : reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 4, 2, false, false, true>);
}

// code: -1 to read x, -2 to read x in rows that start anywhere.
template <typename T>
const void *rms_grad_kernel(int nv, int code, bool full)
{
    if (code == -2)
        return nv == 1   ? reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 1, -1, true, false, false>)
               : nv == 2 ? reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 2, -1, true, false, false>)
                         : reinterpret_cast<void *>(&taco_rms_grad_kernel<T, 4, -1, true, false, false>);
    return code < 0    ? rms_grad_kernel<T, -1>(nv, full)
           : code == 0 ? rms_grad_kernel<T, 0>(nv, full)
           : code == 1 ? rms_grad_kernel<T, 1>(nv, full)
                       : rms_grad_kernel<T, 2>(nv, full);
}

// Kernel and shape; false where the rows do not fit shared memory.
template <typename T>
bool rms_grad_shared(RmsGradArgs *a, bool direct, int sms, cudaStream_t stream, cudaError_t *result)
{
    const int64_t C = a->hidden;
    const bool records = !a->x, odd = C % 8 != 0;
    if (C > 32 * kRmsGradThreads || row_vectors(C) > 4 * kRmsGradThreads)
        return false;
    const int vectors = row_vectors(C), nv = vectors <= 32 ? 1 : vectors <= 64 ? 2 : 4;
    int warps = (vectors + 32 * nv - 1) / (32 * nv);
    int groups = row_groups(a->rows, warps, kRmsGradThreads, sms);
    const size_t weight = 32 * static_cast<size_t>(vectors);
    const size_t place = static_cast<size_t>(1 + !records + (!direct && a->dsummed)) * nv * warps * 256 * sizeof(T) +
                         (records ? (C / a->block * (a->block + 8) + 8 + 15) / 16 * 16 : 0);
    // fewer groups where their rows do not fit, with records three of each
    while (groups > 1 && (weight + groups * place > max_shared<T>(180) || (records && ring_stages(weight, groups * place) < 3)))
        groups--;
    const size_t stage = groups * place;
    int stages = std::max(ring_stages(weight, stage, max_shared<T>(180)), records ? std::min(ring_stages(weight, stage), 3) : 1);
    const size_t smem = weight + std::max<size_t>(stages * stage, groups > 1 ? weight * groups : 0);
    if (smem > kMaxShared || (records && stages < 3))
        return false;
    a->nparts = shifted_grid((a->rows + groups - 1) / groups, groups, odd, std::min(sms, kMaxColumnParts));
    void *p[] = {a, &warps, &groups, &stages};
    *result = launch_kernel(direct ? rms_grad_direct_kernel<T>(a->code)
                                   : rms_grad_kernel<T>(nv, records ? a->code : odd ? -2 : -1, C == warps * nv * 256),
                            a->nparts, warps * groups * 32, smem, stream, p);
    return true;
}

template <typename T>
cudaError_t rms_grad_any(RmsGradArgs *a, int sms, cudaStream_t stream)
{
    cudaError_t result;
    if (rms_grad_shared<T>(a, false, sms, stream, &result))
        return result;
    // (all rows that do not fit have four vectors a lane)
    if (!a->x && a->dsummed && rms_grad_shared<T>(a, true, sms, stream, &result))
        return result;
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

template <typename T>
cudaError_t init_rms_grad_type()
{
    for (int nv = 1; nv <= 4; nv *= 2)
        for (int code = -2; code < 3; code++)
            for (int full = 0; full < 2; full++) {
                const cudaError_t e = cudaFuncSetAttribute(rms_grad_kernel<T>(nv, code, full), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           static_cast<int>(kMaxShared));
                if (e != cudaSuccess)
                    return e;
            }
    for (int code = 0; code < 3; code++) {
        const cudaError_t e = cudaFuncSetAttribute(rms_grad_direct_kernel<T>(code), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kMaxShared));
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t init_rms_grad()
{
    cudaError_t e = init_rms_grad_type<__nv_bfloat16>();
    if (e == cudaSuccess)
        e = init_rms_grad_type<__half>();
    return e == cudaSuccess ? init_rms_grad_type<float>() : e;
}

cudaError_t launch_rms_grad(int dtype, RmsGradArgs *a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? rms_grad_any<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? rms_grad_any<__half>(a, sms, stream)
                               : rms_grad_any<float>(a, sms, stream);
}

}  // namespace taco
