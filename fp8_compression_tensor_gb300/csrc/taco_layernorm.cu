// taco_layernorm.cu -- layer norm with 8-bit checkpoints of the normalised
// input, for GB300 (sm_103a).
//
// Forward, per row of C elements: h = x (or round(x + residual)),
//   mu = sum h / C,  v = sum (h - mu)^2 / C,  rstd = 1 / sqrt(v + eps),
//   xhat = (h - mu) rstd,  y = xhat weight + bias,
// and optionally the records of xhat (taco_train.cuh).  Statistics are
// binary32, the variance from the centred values (a second pass), so a large
// mean costs no precision.
#include "taco_norm.cuh"

namespace taco {
namespace {

// ---------------------------------------------------------------------------
// Odd widths too large for shared memory: one CTA per row, element by element
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
    }
}

// ---------------------------------------------------------------------------
// Widths of whole vectors of eight: rows in registers
// ---------------------------------------------------------------------------

// Rows of whole vectors that are too wide for registers: a CTA a row, two
// vectors a lane at a time, the row read three times (from L1 and L2 after the
// first).
constexpr int kWideThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kWideThreads) taco_norm_wide_kernel(NormArgs a)
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
        // f(c) for the lane's vectors, c their first column
        auto each = [&](auto f) {
            for (int64_t base = warp * 512; base < C; base += kWideThreads * 16)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    if (base + j * 256 + lane * 8 < C)
                        f(base + j * 256 + lane * 8);
        };
        float2 total = both(0.f);
        each([&](int64_t c) {
            const F8 h = load(c, true);
#pragma unroll
            for (int i = 0; i < 4; i++)
                total = add2(total, h.v[i]);
        });
        const float mean = cta_sum(total.x + total.y, part) / static_cast<float>(C);
        float2 squares = both(0.f);
        each([&](int64_t c) {
            const F8 h = load(c, false);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 v = add2(h.v[i], both(-mean));
                squares = fma2(v, v, squares);
            }
        });
        const float rstd = inv_sqrt(cta_sum(squares.x + squares.y, part) / static_cast<float>(C) + a.eps);
        if (threadIdx.x == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        for (int64_t base = warp * 512; base < C; base += kWideThreads * 16) {
            F8 h[2];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int64_t c = base + j * 256 + lane * 8;
                if (c < C) {
                    h[j] = load(c, false);
                    F8 y;
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        y.v[i] = h[j].v[i] = mul2(add2(h[j].v[i], both(-mean)), both(rstd));
                    if (a.weight) {
                        const F8 w = load_param_f8(a.weight, a.param_dtype, c);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            y.v[i] = mul2(y.v[i], w.v[i]);
                    }
                    if (a.bias) {
                        const F8 b = load_param_f8(a.bias, a.param_dtype, c);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            y.v[i] = add2(y.v[i], b.v[i]);
                    }
                    store_raw8(static_cast<T *>(a.y) + row * C + c, pack<T>(y));
                }
            }
            if (a.packed) {
                const int left = static_cast<int>(C - base < 512 ? C - base : 512), col[2] = {lane * 8, 256 + lane * 8};
                uint8_t *to = a.packed + (row * C + base) / a.block * (a.block + 8);
                if (a.code == 0)
                    write_records<2, 0>(h, col, left, to, a.block);
                else if (a.code == 1)
                    write_records<2, 1>(h, col, left, to, a.block);
                else
                    write_records<2, 2>(h, col, left, to, a.block);
            }
        }
    }
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
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group, step = static_cast<int64_t>(gridDim.x) * groups;
    if (warp == 0 && lane < 2 && first + lane * step < a.rows) {
        // the group's first rows on their way to L2 while the kernel before still runs (16384 x 8192 bf16 85 -> 82 us)
        bulk_prefetch_l2(x + (first + lane * step) * C, C * static_cast<int>(sizeof(T)));
        if (res)
            bulk_prefetch_l2(res + (first + lane * step) * C, C * static_cast<int>(sizeof(T)));
    }
    grid_dependency_wait();
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
            uint32_t to = ring_at + static_cast<uint32_t>(stage * row_units * unit);
            auto piece = [&](const T *src) {
#pragma unroll
                for (int j = 0; j < NV; j++)
#pragma unroll
                    for (int k = 0; k < kUnits; k++, to += unit)
                        if (FULL || col[j] < C)
                            copy16<T>(to, reinterpret_cast<const uint4 *>(src + row * C + col[j]) + k);
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
        if (a.packed) {
            uint8_t *to = a.packed + row * (C / a.block) * (a.block + 8);
            if (a.code == 0)
                write_records<NV, 0>(h, col, C, to, a.block);
            else if (a.code == 1)
                write_records<NV, 1>(h, col, C, to, a.block);
            else
                write_records<NV, 2>(h, col, C, to, a.block);
        }
    }
}

// ---------------------------------------------------------------------------
// Widths that are no multiple of 8 (rows that start at any element)
// ---------------------------------------------------------------------------

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
cudaError_t norm_vectors(const NormArgs &a, int sms, cudaStream_t stream)
{
    NormArgs args = a;
    const int nv = lane_vectors(a.hidden);
    int warps = static_cast<int>((a.hidden + 256 * nv - 1) / (256 * nv));
    int groups = row_groups(a.rows, warps, kNormThreads, sms);
    const size_t place = static_cast<size_t>(a.residual ? 2 : 1) * nv * warps * 256 * sizeof(T);
    while (groups > 1 && 8 * static_cast<size_t>(a.hidden) + groups * place > max_shared<T>(196))
        groups--;
    const int threads = warps * groups * 32;
    const int64_t ctas = (a.rows + groups - 1) / groups;
    const size_t stage = groups * place;
    // (the widest binary32 rows with a residual leave no room for the parameters)
    const bool staged = ctas > sms && (a.weight || a.bias) && 8 * static_cast<size_t>(a.hidden) + stage <= kMaxShared;
    const size_t params = staged ? 8 * static_cast<size_t>(a.hidden) : 0;
    int stages = ring_stages(params, stage, max_shared<T>(196));
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
    if (fits_registers(a.hidden) && a.hidden % 8 && norm_odd<T>(a, sms, stream, &result))
        return result;
    if (a.hidden % 8 == 0) {
        NormArgs args = a;
        void *p[] = {&args};
        return launch_kernel(reinterpret_cast<void *>(&taco_norm_wide_kernel<T>), row_grid(a.rows, sms, 4), kWideThreads, 0, stream, p);
    }
    NormArgs args = a;
    void *p[] = {&args};
    return launch_kernel(reinterpret_cast<void *>(&taco_norm_any_kernel<T>), row_grid(a.rows, sms, 8), kRowThreads, 0,
                         stream, p);
}

template <typename T>
cudaError_t init_norm_type()
{
    for (int nv = 1; nv <= 4; nv *= 2)
        for (int i = 0; i < 5; i++) {
            const cudaError_t e = cudaFuncSetAttribute(i < 4 ? norm_kernel<T>(nv, i & 1, i & 2) : norm_odd_kernel<T>(nv),
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxShared));
            if (e != cudaSuccess)
                return e;
        }
    return cudaSuccess;
}

}  // namespace

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

}  // namespace taco
