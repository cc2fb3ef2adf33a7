// taco_weight_grad.cu -- weight gradient of a linear layer whose input was
// kept as an 8-bit checkpoint, for GB300 (sm_103a).
//
//   dW[m, n] = scale[n] sum_r dY[r, m] X[r, n] + dy_sum[m] shift[n]  [+ dW before]
//
// with X the values of the records and dY the bf16 gradient of the layer's
// output.  scale and shift (a layer norm's weight and bias) turn the records
// of the normalised input xhat into those of the norm's output xhat scale +
// shift without decoding them twice: both act per column n, so they leave the
// sum over rows and join the epilogue; dy_sum[m] = sum_r dY[r, m] is the
// layer's bias gradient.
//
// The tensor-core kernel.  A pair of CTAs (a cluster of two) computes a 256 x
// 256 tile of dW with tcgen05.mma.cta_group::2 (M = 256, N = 256, K = 16 rows of
// dY and X per instruction).  Both operands are MN-major: dY's rows hold M
// contiguously and come by TMA (128-byte swizzle); X's rows hold N contiguously
// and are decoded by four warps from record bytes to bf16 in the same layout,
// each CTA decoding the 128 columns that it feeds to the pair.  The pair halves
// the decoding per product: a single CTA with M = 128 would decode each code for
// half as many products.
//
// Binary32 sums.  A tensor-core accumulator cuts (rather than rounds) each
// addition, which biases a long sum: against 64 bits a bf16 product with f32
// output is off by 2.3e-7 (relative 2-norm) over 1024 rows, but by 3.2e-6 over
// 8192.  So an accumulator runs over at most kChunkRows rows; eight epilogue
// warps then add it to the tile's sums, 128 registers a thread, while the next
// chunk runs into the other half of tensor memory.
//
// Roles (512 threads): warp 0 loads dY, warp 1 of the even CTA issues the
// products, warp 2 owns tensor memory, warps 4-7 decode, warps 8-15 add up and
// write.
#include <algorithm>
#include <climits>

#include "taco_host.h"
#include "taco_kernels.h"
#include "taco_tcgen05.cuh"
#include "taco_train.cuh"

namespace taco {
namespace {

constexpr int kTile = 64, kDepth = 16;

__device__ __forceinline__ void finish_element(const WeightGradArgs &a, int64_t m, int64_t n, float v)
{
    if (a.scale)
        v *= load_param(a.scale, a.param_dtype, n);
    if (a.shift)
        v = fmaf(a.dy_sum[m], load_param(a.shift, a.param_dtype, n), v);
    const int64_t i = m * a.hidden + n;
    if (a.accumulate)
        v += load_param(a.dw, a.dtype, i);
    store_param(a.dw, a.dtype, i, v);
}

// Four columns of row m; sum = dy_sum[m].
__device__ __forceinline__ void finish4(const WeightGradArgs &a, int64_t m, int64_t n, float sum, float4 v)
{
    if (a.scale) {
        v.x *= load_param(a.scale, a.param_dtype, n);
        v.y *= load_param(a.scale, a.param_dtype, n + 1);
        v.z *= load_param(a.scale, a.param_dtype, n + 2);
        v.w *= load_param(a.scale, a.param_dtype, n + 3);
    }
    if (a.shift) {
        v.x = fmaf(sum, load_param(a.shift, a.param_dtype, n), v.x);
        v.y = fmaf(sum, load_param(a.shift, a.param_dtype, n + 1), v.y);
        v.z = fmaf(sum, load_param(a.shift, a.param_dtype, n + 2), v.z);
        v.w = fmaf(sum, load_param(a.shift, a.param_dtype, n + 3), v.w);
    }
    const int64_t i = m * a.hidden + n;
    if (a.dtype == kTypeF32) {
        float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(a.dw) + i);
        if (a.accumulate) {
            const float4 w = *to;
            v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
        }
        *to = v;
    } else {
        uint2 *to = reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.dw) + i);
        if (a.accumulate) {
            const uint2 w = *to;
            v = make_float4(v.x + __uint_as_float(w.x << 16), v.y + __uint_as_float(w.x & 0xffff0000u),
                            v.z + __uint_as_float(w.y << 16), v.w + __uint_as_float(w.y & 0xffff0000u));
        }
        *to = make_uint2(float2_to_bf16x2(v.x, v.y), float2_to_bf16x2(v.z, v.w));
    }
}

// ---------------------------------------------------------------------------
// Output widths that are no multiple of 8 (dY's rows are then not 16-byte
// aligned, which TMA needs): CUDA cores
// ---------------------------------------------------------------------------

// 64 x 64 tiles of dW, 4 x 4 values a thread.
__global__ void __launch_bounds__(256) taco_weight_grad_any_kernel(WeightGradArgs a)
{
    __shared__ float sa[kDepth][kTile], sb[kDepth][kTile];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t across = (a.hidden + kTile - 1) / kTile;
    const int64_t m0 = blockIdx.x / across * kTile, n0 = blockIdx.x % across * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const __nv_bfloat16 *dy = static_cast<const __nv_bfloat16 *>(a.dy);
    float acc[4][4] = {};
    for (int64_t r0 = 0; r0 < a.rows; r0 += kDepth) {
        __syncthreads();
        for (int i = threadIdx.x; i < kDepth * kTile; i += 256) {
            const int64_t r = r0 + i / kTile, m = m0 + i % kTile, n = n0 + i % kTile;
            sa[i / kTile][i % kTile] = r < a.rows && m < a.out ? __bfloat162float(dy[r * a.out + m]) : 0.f;
            sb[i / kTile][i % kTile] =
                r < a.rows && n < a.hidden ? record_value(a.packed, r * a.hidden + n, a.block, a.code) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; k++) {
            float x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[j] = sa[k][ty * 4 + j];
                y[j] = sb[k][tx * 4 + j];
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
        }
    }
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++)
            if (m0 + ty * 4 + i < a.out && n0 + tx * 4 + j < a.hidden)
                finish_element(a, m0 + ty * 4 + i, n0 + tx * 4 + j, acc[i][j]);
}

// ---------------------------------------------------------------------------
// Tensor-core kernel
// ---------------------------------------------------------------------------

constexpr int kPairM = 256, kPairN = 256;     // tile of a CTA pair; each CTA holds 128 rows of A and of B
constexpr int kStageRows = 64;                // rows of dY and X per pipeline stage
constexpr int kChunkRows = 1024;              // rows per tensor-core accumulation
constexpr int kStages = 5, kRawStages = 5;
constexpr int kOperandBytes = 128 * kStageRows * 2;             // one CTA's A or B of a stage
constexpr int kHalfBytes = 64 * kStageRows * 2;                 // 64 columns of it
constexpr int kRawWarpBytes = 16 * 128 + 16 * 4 * 8;            // a decoder warp's 16 rows: codes, (alpha, s) pairs
constexpr int kRawBytes = 4 * kRawWarpBytes;
constexpr int kWgThreads = 512;
constexpr size_t kWgSmem = 1024 + static_cast<size_t>(kStages) * 2 * kOperandBytes + kRawStages * kRawBytes + 512;
constexpr uint32_t kIdesc = mma_idesc_bf16_f32(kPairM, kPairN) | (1u << 15) | (1u << 16);   // A and B MN-major

struct WgBarriers {
    uint64_t a_full[kStages];     // this CTA's dY tile has landed
    uint64_t full[kStages];       // even CTA: both CTAs' A and B of the stage are ready
    uint64_t empty[kStages];      // the stage's products are done
    uint64_t acc_full[2];         // a chunk's accumulator is complete
    uint64_t acc_empty[2];        // even CTA: both CTAs have read the accumulator
    uint32_t tmem;
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The even CTA's address of this CTA's shared-memory address.
__device__ __forceinline__ uint32_t in_even_cta(uint32_t addr)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ void cluster_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded wait for a barrier that the other CTA's threads arrive on too.
__device__ __forceinline__ bool cluster_wait(uint32_t bar, uint32_t parity, uint32_t *fault)
{
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(TACO_WAIT_HINT_NS)
            : "memory");
        if (ok)
            return true;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            atomicOr(fault, kFaultWeightGrad);
            return false;
        }
    }
}


// MN-major operand in the 128-byte swizzled layout: rows of 64 MN-elements,
// 8-row groups 1024 bytes apart, blocks of 64 MN-elements kHalfBytes apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((kHalfBytes >> 4) & 0x3FFF) << 16;
    d |= static_cast<uint64_t>((1024u >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(kIdesc), "r"(accumulate)
        : "memory");
}

// One arrival on the barrier at this offset in both CTAs once the pair's products so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Copies 8 bytes, or zeros where `valid` is false (src is then not read).
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(valid ? 8 : 0) : "memory");
}

// Two codes (low 16 bits of `pair`) times f, rounded to bf16 (exact for a power of two).
template <int CODE>
__device__ __forceinline__ uint32_t decode2(uint32_t pair, float f)
{
    const float2 v = mul2(CODE == 0 ? e4m3x2_to_float2(pair) : e5m2x2_to_float2(pair), make_float2(f, f));
    return float2_to_bf16x2(v.x, v.y);
}

template <int CODE>
__device__ __forceinline__ uint4 decode8(uint2 c, float f)
{
    if (CODE == 2) {
        const float2 f2 = make_float2(f, f);
        float2 a, b, d, e;
        int8x4_to_float(c.x, a, b);
        int8x4_to_float(c.y, d, e);
        a = mul2(a, f2), b = mul2(b, f2), d = mul2(d, f2), e = mul2(e, f2);
        return make_uint4(float2_to_bf16x2(a.x, a.y), float2_to_bf16x2(b.x, b.y), float2_to_bf16x2(d.x, d.y),
                          float2_to_bf16x2(e.x, e.y));
    }
    return make_uint4(decode2<CODE>(c.x & 0xffffu, f), decode2<CODE>(c.x >> 16, f), decode2<CODE>(c.y & 0xffffu, f),
                      decode2<CODE>(c.y >> 16, f));
}

// Tiles of the grid's work: unit -> (split, tile row, tile column), columns fastest.
struct WgPlan {
    int64_t units;
    int tiles_m, tiles_n, stages_total, splits;
    __device__ void at(int64_t u, int &m0, int &n0, int &split, int &first, int &count) const
    {
        const int64_t tiles = static_cast<int64_t>(tiles_m) * tiles_n;
        split = static_cast<int>(u / tiles);
        const int64_t t = u - split * tiles;
        m0 = static_cast<int>(t / tiles_n) * kPairM;
        n0 = static_cast<int>(t % tiles_n) * kPairN;
        first = static_cast<int>(static_cast<int64_t>(stages_total) * split / splits);
        count = static_cast<int>(static_cast<int64_t>(stages_total) * (split + 1) / splits) - first;
    }
};

template <int CODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgThreads, 1)
taco_weight_grad_kernel(const __grid_constant__ CUtensorMap map_dy, WeightGradArgs a, WgPlan plan, uint32_t *fault)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) WgBarriers bars;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t raw = base + kStages * 2 * kOperandBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int64_t first_unit = blockIdx.x >> 1, step_units = gridDim.x >> 1;
    auto bar = [](uint64_t &b) { return smem_addr(&b); };

    grid_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(bar(bars.a_full[s]), 1);
            mbar_init(bar(bars.full[s]), 8);       // four decoder warps of each CTA
            mbar_init(bar(bars.empty[s]), 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(bar(bars.acc_full[b]), 1);
            mbar_init(bar(bars.acc_empty[b]), 16); // eight epilogue warps of each CTA
        }
        fence_mbar_init();
        prefetch_tmap(&map_dy);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&bars.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before_sync();
    cta_barrier();
    cluster_barrier();
    tc_fence_after_sync();
    const uint32_t tmem = bars.tmem;
    grid_dependency_wait();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0 && lane == 0) {
            // dY: two boxes of 64 columns by 64 rows a stage
            int64_t it = 0;
            bool ok = true;
            for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
                int m0, n0, split, first, count;
                plan.at(u, m0, n0, split, first, count);
                const int x = m0 + static_cast<int>(rank) * 128;
                for (int k = first; k < first + count; k++, it++) {
                    const int s = static_cast<int>(it % kStages);
                    if (it >= kStages && !mbar_wait_bounded_thread(bar(bars.empty[s]), static_cast<uint32_t>(it / kStages - 1) & 1u,
                                                                   fault, kFaultWeightGrad)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = base + s * 2 * kOperandBytes;
                    mbar_arrive_expect_tx(bar(bars.a_full[s]), kOperandBytes);
                    tma_load_2d(dst, &map_dy, x, k * kStageRows, bar(bars.a_full[s]));
                    tma_load_2d(dst + kHalfBytes, &map_dy, x + 64, k * kStageRows, bar(bars.a_full[s]));
                }
            }
            // no copy may land after the CTA is gone
            for (int64_t i = it > kStages ? it - kStages : 0; i < it; i++)
                mbar_wait_bounded_thread(bar(bars.a_full[i % kStages]), static_cast<uint32_t>(i / kStages) & 1u, fault,
                                         kFaultWeightGrad);
        } else if (warp == 1 && lane == 0 && rank == 0) {
            int64_t it = 0, chunk = 0;
            bool ok = true;
            for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
                int m0, n0, split, first, count;
                plan.at(u, m0, n0, split, first, count);
                for (int k = 0; k < count && ok; chunk++) {
                    const int b = static_cast<int>(chunk & 1);
                    if (chunk >= 2 && !cluster_wait(bar(bars.acc_empty[b]), static_cast<uint32_t>((chunk >> 1) - 1) & 1u, fault)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const int end = min(count, k + kChunkRows / kStageRows);
                    for (const int begin = k; k < end; k++, it++) {
                        const int s = static_cast<int>(it % kStages);
                        if (!cluster_wait(bar(bars.full[s]), static_cast<uint32_t>(it / kStages) & 1u, fault)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t sa = base + s * 2 * kOperandBytes;
#pragma unroll
                        for (int j = 0; j < kStageRows / 16; j++)
                            pair_mma(tmem + b * kPairN, mn_desc(sa + j * 2048), mn_desc(sa + kOperandBytes + j * 2048),
                                     k > begin || j > 0);
                        pair_commit(bar(bars.empty[s]));
                    }
                    if (ok)
                        pair_commit(bar(bars.acc_full[b]));
                }
            }
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        // Decoders: warp d takes rows 16 d .. 16 d + 15 of every stage; lane l the
        // codes 8 (l % 16) .. of rows l / 16, l / 16 + 2, ...
        const int d = warp - 4, B = a.block, sub = lane >> 4, col = (lane & 15) * 8;
        const int per_row = B < 128 ? 128 / B : 1;             // blocks of a row's 128 columns
        const int64_t pitch = a.hidden / B * (B + 8);
        const uint32_t my_raw = raw + d * kRawWarpBytes;
        const uint32_t swz = static_cast<uint32_t>(lane & 7);
        const uint32_t full0 = in_even_cta(bar(bars.full[0]));
        // Producer position (the record bytes) and consumer position.
        int64_t pu = first_unit, pit = 0;
        int pk = 0, pcount = 0, pn = 0, pfirst = 0;
        auto enter = [&]() {
            if (pu < plan.units) {
                int m0, split;
                plan.at(pu, m0, pn, split, pfirst, pcount);
                pn += static_cast<int>(rank) * 128;
            }
        };
        auto produce = [&]() {
            while (pu < plan.units && pk == pcount) {
                pu += step_units;
                pk = 0;
                enter();
            }
            if (pu < plan.units) {
                const uint32_t slot = my_raw + static_cast<uint32_t>(pit % kRawStages) * kRawBytes;
                const int64_t r0 = static_cast<int64_t>(pfirst + pk) * kStageRows + d * 16;
                const int64_t n = pn + col;
                const uint8_t *src = a.packed + r0 * pitch + n / B * (B + 8) + n % B;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int row = 2 * j + sub;
                    const bool valid = n < a.hidden && r0 + row < a.rows;
                    copy8(slot + row * 128 + col, valid ? src + row * pitch : a.packed, valid);
                }
                for (int i = lane; i < 16 * per_row; i += 32) {
                    const int row = i / per_row;
                    const int64_t nb = pn + static_cast<int64_t>(i % per_row) * B;
                    const bool valid = nb < a.hidden && r0 + row < a.rows;
                    copy8(slot + 2048 + i * 8, valid ? a.packed + (r0 + row) * pitch + nb / B * (B + 8) + B : a.packed, valid);
                }
                pk++;
                pit++;
            }
            cp_async_commit();
        };
        enter();
        for (int i = 0; i < kRawStages - 1; i++)
            produce();
        int64_t it = 0;
        bool ok = true;
        for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
            int m0, n0, split, first, count;
            plan.at(u, m0, n0, split, first, count);
            for (int k = 0; k < count; k++, it++) {
                const int s = static_cast<int>(it % kStages);
                __syncwarp();                                  // every lane has read the slot that produce() refills
                produce();
                cp_async_wait<kRawStages - 1>();
                __syncwarp();
                if (it >= kStages && !mbar_wait_bounded(bar(bars.empty[s]), static_cast<uint32_t>(it / kStages - 1) & 1u, fault,
                                                        kFaultWeightGrad)) {
                    ok = false;
                    break;
                }
                const uint32_t slot = my_raw + static_cast<uint32_t>(it % kRawStages) * kRawBytes;
                const uint32_t dst = base + s * 2 * kOperandBytes + kOperandBytes + (col >> 6) * kHalfBytes;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int row = 2 * j + sub, kr = d * 16 + row;
                    const uint2 c = lds64(slot + row * 128 + col);
                    const uint2 meta = lds64(slot + 2048 + (row * per_row + (per_row > 1 ? col / B : 0)) * 8);
                    const float alpha = __uint_as_float(meta.x);
                    float f = __uint_as_float(meta.y);
                    if (alpha != 1.f && f != 0.f)
                        f = __fdiv_rn(f, alpha);
                    sts128(dst + (kr >> 3) * 1024 + (kr & 7) * 128 + ((swz ^ (kr & 7)) << 4), decode8<CODE>(c, f));
                }
                fence_proxy_async_smem();
                if (!mbar_wait_bounded(bar(bars.a_full[s]), static_cast<uint32_t>(it / kStages) & 1u, fault, kFaultWeightGrad)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                if (lane == 0)
                    cluster_arrive(full0 + s * 8);
            }
        }
        cp_async_wait<0>();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // Epilogue: warp w reads lanes 32 (w % 4) .., columns 128 (w / 4 - 2) .. of the accumulators.
        const int quarter = warp & 3, half = (warp - 8) >> 2;
        const uint32_t empty0 = in_even_cta(bar(bars.acc_empty[0]));
        int64_t chunk = 0;
        bool ok = true;
        for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
            int m0, n0, split, first, count;
            plan.at(u, m0, n0, split, first, count);
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; i++)
                acc[i] = 0.f;
            for (int k = 0; k < count; k += kChunkRows / kStageRows, chunk++) {
                const int b = static_cast<int>(chunk & 1);
                if (!mbar_wait_bounded(bar(bars.acc_full[b]), static_cast<uint32_t>(chunk >> 1) & 1u, fault, kFaultWeightGrad)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t src = tmem + (static_cast<uint32_t>(quarter) << 21) + b * kPairN + half * 128;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    uint32_t r[32];
                    tmem_ld32(src + c * 32, r);
                    tmem_ld_wait();
                    tmem_regs_ready(r);
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        acc[c * 32 + i] += __uint_as_float(r[i]);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    cluster_arrive(empty0 + b * 8);
            }
            const int64_t m = m0 + static_cast<int64_t>(rank) * 128 + quarter * 32 + lane;
            if (!ok || m >= a.out)
                continue;
            const int64_t nbase = n0 + half * 128;
            if (plan.splits > 1) {
                float *to = a.parts + (split * a.out + m) * a.hidden + nbase;
#pragma unroll
                for (int i = 0; i < 128; i += 4)
                    if (nbase + i < a.hidden)
                        *reinterpret_cast<float4 *>(to + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
            } else {
                const float sum = a.shift ? a.dy_sum[m] : 0.f;
#pragma unroll
                for (int i = 0; i < 128; i += 4)
                    if (nbase + i < a.hidden)
                        finish4(a, m, nbase + i, sum, make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]));
            }
        }
    }
    tc_fence_before_sync();
    cta_barrier();
    cluster_barrier();
    tc_fence_after_sync();
    __syncwarp();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Adds the splits' sums in order and finishes four columns a thread.
__global__ void __launch_bounds__(256) taco_weight_grad_join_kernel(WeightGradArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t n = a.out * a.hidden;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < n; i += 1024ll * gridDim.x) {
        float4 v = *reinterpret_cast<const float4 *>(a.parts + i);
        for (int s = 1; s < a.splits; s++) {
            const float4 w = *reinterpret_cast<const float4 *>(a.parts + s * n + i);
            v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
        }
        const int64_t m = i / a.hidden;
        finish4(a, m, i - m * a.hidden, a.shift ? a.dy_sum[m] : 0.f, v);
    }
}

const void *wg_kernel(int code)
{
    return code == 0   ? reinterpret_cast<void *>(&taco_weight_grad_kernel<0>)
           : code == 1 ? reinterpret_cast<void *>(&taco_weight_grad_kernel<1>)
                       : reinterpret_cast<void *>(&taco_weight_grad_kernel<2>);
}

cudaError_t launch_pairs(const void *fn, int pairs, cudaStream_t stream, void **args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kWgThreads);
    cfg.dynamicSmemBytes = kWgSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = TACO_PDL ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// The tensor-core kernel's TMA view of dY needs rows of a multiple of 16 bytes.
bool on_tensor_cores(int64_t out) { return out % 8 == 0; }

}  // namespace

cudaError_t init_weight_grad()
{
    cudaError_t e = cudaSuccess;
    for (int code = 0; code < 3 && e == cudaSuccess; code++)
        e = cudaFuncSetAttribute(wg_kernel(code), cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kWgSmem));
    return e;
}

// Splits the rows where the tiles leave CTA pairs (of 76) idle, down to 512 rows a split.
int weight_grad_splits(int64_t rows, int64_t out, int64_t hidden)
{
    if (!on_tensor_cores(out))
        return 1;
    const int64_t tiles = ((out + kPairM - 1) / kPairM) * ((hidden + kPairN - 1) / kPairN);
    if (tiles == 0)
        return 1;
    const int64_t splits = std::min<int64_t>(76 / tiles, rows / 512);
    return static_cast<int>(std::max<int64_t>(splits, 1));
}

bool weight_grad_in_range(int64_t rows, int64_t out, int64_t hidden)
{
    // 32-bit TMA coordinates, whole tiles and stages past the end included
    return rows <= INT32_MAX - 64 && out <= INT32_MAX - 256 && hidden <= INT32_MAX - 256 && (out + kTile - 1) / kTile <= INT32_MAX / ((hidden + kTile - 1) / kTile + 1);
}

cudaError_t launch_weight_grad(const WeightGradArgs &a, uint32_t *fault, int sms, cudaStream_t stream)
{
    WeightGradArgs args = a;
    if (!on_tensor_cores(a.out) || a.rows == 0) {
        void *p[] = {&args};
        const int64_t tiles = (a.hidden + kTile - 1) / kTile * ((a.out + kTile - 1) / kTile);
        return launch_kernel(reinterpret_cast<void *>(&taco_weight_grad_any_kernel), static_cast<int>(tiles), 256, 0, stream, p);
    }
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    cudaError_t e = tensor_map_encoder(&encode);
    if (e != cudaSuccess)
        return e;
    alignas(64) CUtensorMap map;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.out), static_cast<cuuint64_t>(a.rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.out) * 2};
    const cuuint32_t box[2] = {64, kStageRows}, elem_strides[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(a.dy), dims, strides, box, elem_strides,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    WgPlan plan;
    plan.tiles_m = static_cast<int>((a.out + kPairM - 1) / kPairM);
    plan.tiles_n = static_cast<int>((a.hidden + kPairN - 1) / kPairN);
    plan.stages_total = static_cast<int>((a.rows + kStageRows - 1) / kStageRows);
    plan.splits = a.splits;
    plan.units = static_cast<int64_t>(plan.tiles_m) * plan.tiles_n * a.splits;
    void *p[] = {&map, &args, &plan, &fault};
    e = launch_pairs(wg_kernel(a.code), static_cast<int>(std::min<int64_t>(plan.units, sms / 2)), stream, p);
    if (e == cudaSuccess && a.splits > 1) {
        void *q[] = {&args};
        const int64_t want = (a.out * a.hidden + 1023) / 1024;
        e = launch_kernel(reinterpret_cast<void *>(&taco_weight_grad_join_kernel),
                          static_cast<int>(std::min<int64_t>(want, 8ll * sms)), 256, 0, stream, q);
    }
    return e;
}

}  // namespace taco
