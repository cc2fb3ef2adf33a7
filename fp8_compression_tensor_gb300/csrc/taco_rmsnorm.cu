// taco_rmsnorm.cu -- root-mean-square norm with the residual's addition, 8-bit
// checkpoints of the normalised rows and 8-bit outputs, for GB300 (sm_103a).
//
// Per row of C elements: h = x (or round(x + residual)),
//   rstd = 1 / sqrt(sum h^2 / C + eps),  xhat = h rstd,  y = xhat weight,
// y as a tensor or as records, and optionally the records of xhat
// (taco_train.cuh).  Sums are binary32.
#include "taco_rms.cuh"

namespace taco {
namespace {

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

// ---------------------------------------------------------------------------
// Rows whose squares leave binary32
// ---------------------------------------------------------------------------

// Squares that overflowed, or that were flushed (below 2^-149 each), can be seen in a row's rstd where it is not
// between 2^-64 and 2^40.  The loop over the rows keeps the largest of these numbers, which have the order of rstd above
// 2^-64 and lie above kRangeBits for all others.
constexpr uint32_t kRangeFirst = 0x1f800001u, kRangeBits = 0x53800000u - kRangeFirst;   // the bits of 2^-64 and one, of 2^40
__device__ __forceinline__ uint32_t range_bits(float rstd) { return __float_as_uint(rstd) - kRangeFirst; }

// 2^-e for a row whose largest |h| has the bits `top` (bits have the order of their values, a NaN's above all), or 0
// where rstd stays as it is: for infinities and NaN, and for zeros without eps.
__device__ __forceinline__ float row_scale(uint32_t top, float eps)
{
    const uint32_t most = max(top, __float_as_uint(sqrtf(eps)));
    if (most - 1u >= 0x7f7fffffu)
        return 0.f;
    const int e = static_cast<int>(most >> 23);          // 127 more than that of the power of two; 0 for subnormal numbers
    return e < 253 ? __uint_as_float(static_cast<uint32_t>(254 - max(e, 1)) << 23) : 0x1p-126f;
}

// Makes such rows again, of those that a group of `warps` warps (one of `groups` in the CTA) has taken: with squares of
// h 2^-e, 2^e being the power of two at or below max(max|h|, sqrt(eps)).  `sums` has two places a warp, 32 apart.
// It stands behind the loop over the rows and takes the thread's place anew, so that the loop keeps nothing for it: inside
// the loop, ahead of y, it took 4096 x 20480 bf16 from 50.2 to 53.8 us and 8192 x 4097 with a residual from 46.9 to 48.1.
template <typename T, bool ODD>
__device__ __forceinline__ void redo_rows(const RmsArgs &a, int warps, int groups, float *sums)
{
    uint32_t tid, bid;
    asm volatile("mov.u32 %0, %%tid.x;\n\tmov.u32 %1, %%ctaid.x;" : "=r"(tid), "=r"(bid));
    const int lane = tid & 31, group = (tid >> 5) / warps, warp = (tid >> 5) - group * warps;
    const int threads = warps * 32, thread = warp * 32 + lane;
    const int64_t C = a.hidden, step = static_cast<int64_t>(gridDim.x) * groups;
    float *one = sums + group * warps, *two = one + 32;
    auto barrier = [&] {
        if (warps == 1)
            __syncwarp();
        else
            group_barrier(1 + group, threads);
    };
    barrier();   // behind the group's last stores
#pragma unroll 1
    for (int64_t row = ODD ? bid + static_cast<int64_t>(gridDim.x) * group : static_cast<int64_t>(bid) * groups + group; row < a.rows; row += step) {
        if (range_bits(a.rstd[row]) < kRangeBits)
            continue;
        const T *x = static_cast<const T *>(a.x) + row * C, *res = a.residual ? static_cast<const T *>(a.residual) + row * C : nullptr;
        auto h = [&](int64_t c) {
            const float v = to_float(x[c]);
            return res ? to_float(from_float<T>(v + to_float(res[c]))) : v;
        };
        uint32_t top = 0u;
#pragma unroll 1
        for (int64_t c = thread; c < C; c += threads)
            top = max(top, abs_bits(h(c)));
        top = __reduce_max_sync(kFullMask, top);
        barrier();   // all have read the row's rstd, and the sums of the row before
        if (lane == 0)
            one[warp] = __uint_as_float(top);
        barrier();
        const float scale = row_scale(__reduce_max_sync(kFullMask, lane < warps ? __float_as_uint(one[lane]) : 0u), a.eps);
        if (scale == 0.f)
            continue;
        float sq = 0.f;
#pragma unroll 1
        for (int64_t c = thread; c < C; c += threads) {
            const float v = h(c) * scale;
            sq = fmaf(v, v, sq);
        }
        sq = warp_sum(sq);
        if (lane == 0)
            two[warp] = sq;
        barrier();
        sq = warp_sum(lane < warps ? two[lane] : 0.f);
        const float rstd = scale * inv_sqrt(sq / static_cast<float>(C) + a.eps * scale * scale);
        if (thread == 0)
            a.rstd[row] = rstd;
        if (ODD || a.y)
#pragma unroll 1
            for (int64_t c = thread; c < C; c += threads) {
                float v = h(c) * rstd;
                if (a.weight)
                    v *= load_param(a.weight, a.param_dtype, c);
                static_cast<T *>(a.y)[row * C + c] = from_float<T>(v);
            }
#pragma unroll 1
        for (int k = 0; k < 2 && !ODD; k++) {
            uint8_t *to = k ? a.packed_y : a.packed;
#pragma unroll 1
            for (int64_t base = warp * 512; to && base < C; base += warps * 512) {
                F8 u[2] = {};
                const int left = static_cast<int>(C - base < 512 ? C - base : 512), col[2] = {lane * 8, 256 + lane * 8};
#pragma unroll
                for (int j = 0; j < 2; j++)
                    if (col[j] < left) {
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const int64_t c = base + col[j] + i;
                            float v = h(c) * rstd;
                            if (k && a.weight)
                                v *= load_param(a.weight, a.param_dtype, c);
                            (i % 2 ? u[j].v[i / 2].y : u[j].v[i / 2].x) = v;
                        }
                    }
                write_records_of<2>(u, col, left, to + (row * C + base) / a.block * (a.block + 8), a.block, a.code);
            }
        }
    }
}

// The same as a call, which the kernel of rows that start anywhere makes: with its registers the code above took 8192 x
// 4097 to 48.6 us; so it takes 47.1.
template <typename T>
__device__ __noinline__ void call_redo_rows(const void *x, const void *residual, const void *weight, void *y, float *rstd, int64_t rows,
                                            int64_t hidden, float eps, int param_dtype, int warps, int groups, float *sums)
{
    const RmsArgs a{x, residual, weight, y, nullptr, rstd, nullptr, nullptr, rows, hidden, eps, param_dtype, 0, 0};
    redo_rows<T, true>(a, warps, groups, sums);
}

// ---------------------------------------------------------------------------
// Any width: a CTA a row, element by element (no records: those need widths of
// whole blocks)
// ---------------------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(kRowThreads) taco_rms_any_kernel(RmsArgs a)
{
    __shared__ float part[64];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden;
    uint32_t ranges = 0u;
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
        ranges = max(ranges, range_bits(rstd));
    }
    if (ranges >= kRangeBits)
        redo_rows<T, true>(a, kRowThreads / 32, 1, part);
}

// ---------------------------------------------------------------------------
// Widths of whole vectors of eight: a CTA a row, two vectors a lane at a time,
// the row read twice (the second time from L1 and L2)
// ---------------------------------------------------------------------------

constexpr int kWideThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kWideThreads) taco_rms_wide_kernel(RmsArgs a)
{
    __shared__ float part[64];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t C = a.hidden;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t ranges = 0u;
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
        ranges = max(ranges, range_bits(rstd));
    }
    if (ranges >= kRangeBits)
        redo_rows<T, false>(a, kWideThreads / 32, 1, part);
}

// ---------------------------------------------------------------------------
// Rows in registers
// ---------------------------------------------------------------------------

// The layer norm's arrangement: a row's vectors over a group of `warps` warps,
// vector j (of NV) of warp w, lane l being (w NV + j) 32 + l, the CTA's groups on
// rows of their own, rows on their way to shared memory `stages` ahead by
// cp.async, each piece copied by the thread that reads it.  One row sum, one
// barrier.
// STAGED: the weight lies in shared memory.  ODD: rows start anywhere (taco_rms.cuh).  FULL: every lane's every
// vector lies inside the row.
constexpr int kRmsThreads = 768;

template <typename T, int NV, bool STAGED, bool ODD, bool FULL>
__global__ void __launch_bounds__(kRmsThreads, 1) taco_rms_kernel(RmsArgs a, int warps, int groups, int stages)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // weight (STAGED), then the copies
    __shared__ float sums[2][32];
    grid_launch_dependents();
    constexpr int kUnits = sizeof(T) / 2;                 // 16-byte units of eight elements
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / warps, warp = (threadIdx.x >> 5) - group * warps;
    const int C = static_cast<int>(a.hidden), unit = blockDim.x * 16, vectors = row_vectors(C);
    const int shift = ODD ? static_cast<int>(blockIdx.x * a.hidden & 7) : 0;
    float *sparam = reinterpret_cast<float *>(dynamic);
    uint8_t *ring = dynamic + (STAGED ? 32 * vectors : 0) + threadIdx.x * 16;
    const uint32_t ring_at = smem_addr(ring);
    const int row_units = (a.residual ? 2 : 1) * NV * kUnits;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
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
        bulk_prefetch_l2(x + (first + lane * step) * C, C * static_cast<int>(sizeof(T)));
        if (res)
            bulk_prefetch_l2(res + (first + lane * step) * C, C * static_cast<int>(sizeof(T)));
    }
    grid_dependency_wait();
    const int64_t end = a.rows * a.hidden * static_cast<int>(sizeof(T));   // of the tensors, in bytes
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            // the tensors' last vector may end behind them
            const bool whole = !ODD || (row * C - shift + 8 * vectors) * static_cast<int>(sizeof(T)) <= end;
            uint32_t to = ring_at + static_cast<uint32_t>(stage * row_units * unit);
            auto piece = [&](const T *src) {
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
            piece(x);
            if (res)
                piece(res);
        }
        copies_issued();
    };
    for (int i = 0; i < stages - 1; i++)
        copy_row(first + i * step, i);
    if (STAGED) {
        stage_shifted<ODD>(sparam, a.weight, a.param_dtype, vectors, shift, C, 1.f);
        __syncthreads();
    }
    auto weight = [&](int j) {
        if (STAGED)
            return load_shifted(sparam, v0 + 32 * j, vectors);
        return ODD ? load_param_edge(a.weight, a.param_dtype, col[j], C, 1.f) : load_param_f8(a.weight, a.param_dtype, col[j]);
    };
    const float fc = static_cast<float>(C);
    int stage = 0, fill = stages - 1;
    uint32_t side = 0;
    uint32_t ranges = 0u;
    for (int64_t row = first; row < a.rows; row += step, side ^= 1u) {
        copy_row(row + (stages - 1) * step, fill);
        fill = fill + 1 == stages ? 0 : fill + 1;
        copies_landed(stages - 1);
        uint8_t *mine = ring + static_cast<size_t>(stage) * row_units * unit;
        stage = stage + 1 == stages ? 0 : stage + 1;
        if (ODD && edges) {
#pragma unroll
            for (int j = 0; j < NV; j++)
                if (col[j] < C && at_edge(col[j], C))
                    clear_edge<T>(mine + j * kUnits * unit, res ? 2 : 1, NV * kUnits * unit, unit, col[j], C);
        }
        F8 h[NV];
        float2 squares = both(0.f);
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
                    store_vector<T, ODD>(static_cast<T *>(a.summed) + row * C, h[j], col[j], C);
                    h[j] = unpack(pack<T>(h[j]));
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
                    squares = fma2(h[j].v[i], h[j].v[i], squares);
            }
        // `sums` alternates between two sets, so a set is written again only behind the next row's barrier
        const float sq = group_sum(warp_sum(squares.x + squares.y), sums[side] + group * warps, group, warp, warps);
        const float rstd = inv_sqrt(sq / fc + a.eps);
        if (warp == 0 && lane == 0)
            a.rstd[row] = rstd;
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    h[j].v[i] = mul2(h[j].v[i], both(rstd));
            }
        if (!ODD && a.packed)
            write_records_of<NV>(h, col, C, a.packed + row * (C / a.block) * (a.block + 8), a.block, a.code);
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (FULL || col[j] < C) {
                if (STAGED || a.weight) {
                    const F8 w = weight(j);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        h[j].v[i] = mul2(h[j].v[i], w.v[i]);
                }
                if (ODD || a.y)
                    store_vector<T, ODD>(static_cast<T *>(a.y) + row * C, h[j], col[j], C);
            }
        if (!ODD && a.packed_y)
            write_records_of<NV>(h, col, C, a.packed_y + row * (C / a.block) * (a.block + 8), a.block, a.code);
        ranges = max(ranges, range_bits(rstd));
    }
    if (ranges >= kRangeBits) {
        if (ODD)
            call_redo_rows<T>(a.x, a.residual, a.weight, a.y, a.rstd, a.rows, a.hidden, a.eps, a.param_dtype, warps, groups, sums[0]);
        else
            redo_rows<T, false>(a, warps, groups, sums[0]);
    }
}

template <typename T, bool STAGED>
const void *rms_kernel(int nv, bool odd, bool full)
{
    if (odd)
        return nv == 1   ? reinterpret_cast<void *>(&taco_rms_kernel<T, 1, STAGED, true, false>)
               : nv == 2 ? reinterpret_cast<void *>(&taco_rms_kernel<T, 2, STAGED, true, false>)
                         : reinterpret_cast<void *>(&taco_rms_kernel<T, 4, STAGED, true, false>);
    return nv == 1   ? reinterpret_cast<void *>(&taco_rms_kernel<T, 1, STAGED, false, false>)
           : nv == 2 ? reinterpret_cast<void *>(&taco_rms_kernel<T, 2, STAGED, false, false>)
           : full    ? reinterpret_cast<void *>(&taco_rms_kernel<T, 4, STAGED, false, true>)
                     : reinterpret_cast<void *>(&taco_rms_kernel<T, 4, STAGED, false, false>);
}

template <typename T>
const void *rms_kernel(int nv, bool staged, bool odd, bool full)
{
    return staged ? rms_kernel<T, true>(nv, odd, full) : rms_kernel<T, false>(nv, odd, full);
}

// Vectors that a CTA's warps hold, four a lane.
constexpr int kRmsVectors = kRmsThreads * 4;

template <typename T>
bool rms_registers(const RmsArgs &a, int sms, cudaStream_t stream, cudaError_t *result)
{
    if (a.hidden > 8 * kRmsVectors || row_vectors(a.hidden) > kRmsVectors)
        return false;
    RmsArgs args = a;
    const int vectors = row_vectors(a.hidden), nv = vectors <= 32 ? 1 : vectors <= 64 ? 2 : 4;
    int warps = (vectors + 32 * nv - 1) / (32 * nv);
    int groups = row_groups(a.rows, warps, kRmsThreads, sms);
    const size_t place = static_cast<size_t>(a.residual ? 2 : 1) * nv * warps * 256 * sizeof(T), params = 32 * static_cast<size_t>(vectors);
    while (groups > 1 && params + groups * place > max_shared<T>(196))
        groups--;
    const size_t stage = groups * place;
    const int64_t ctas = (a.rows + groups - 1) / groups;
    // The weight is staged while the rows are on their way; only a single wide row a CTA reads it faster where it is used (2 x
    // 16384: 3.1 us against 3.7; 4 x 4096 the other way round, 2.7 against 2.3, 1023 x 2055 f32 6.9 against 6.0).
    const bool staged = (ctas > sms || groups > 1 || a.hidden <= 8192) && a.weight && params + stage <= kMaxShared;
    int stages = ring_stages(staged ? params : 0, stage, max_shared<T>(196));
    void *p[] = {&args, &warps, &groups, &stages};
    *result = launch_kernel(rms_kernel<T>(nv, staged, a.hidden % 8 != 0, a.hidden == warps * nv * 256), shifted_grid(ctas, groups, a.hidden % 8 != 0, sms),
                            warps * groups * 32, (staged ? params : 0) + stages * stage, stream, p);
    return true;
}

template <typename T>
cudaError_t rms_any(const RmsArgs &a, int sms, cudaStream_t stream)
{
    cudaError_t result;
    if (rms_registers<T>(a, sms, stream, &result))
        return result;
    RmsArgs args = a;
    void *p[] = {&args};
    if (a.hidden % 8 == 0)
        return launch_kernel(reinterpret_cast<void *>(&taco_rms_wide_kernel<T>), row_grid(a.rows, sms, 4), kWideThreads, 0, stream, p);
    return launch_kernel(reinterpret_cast<void *>(&taco_rms_any_kernel<T>), row_grid(a.rows, sms, 8), kRowThreads, 0, stream, p);
}

template <typename T>
cudaError_t init_rms_type()
{
    for (int nv = 1; nv <= 4; nv *= 2)
        for (int i = 0; i < 8; i++) {
            const cudaError_t e = cudaFuncSetAttribute(rms_kernel<T>(nv, i & 1, i & 2, i & 4), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(kMaxShared));
            if (e != cudaSuccess)
                return e;
        }
    return cudaSuccess;
}

}  // namespace

cudaError_t init_rms()
{
    cudaError_t e = init_rms_type<__nv_bfloat16>();
    if (e == cudaSuccess)
        e = init_rms_type<__half>();
    return e == cudaSuccess ? init_rms_type<float>() : e;
}

cudaError_t launch_rms(int dtype, const RmsArgs &a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? rms_any<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? rms_any<__half>(a, sms, stream)
                               : rms_any<float>(a, sms, stream);
}

}  // namespace taco
