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
// and are decoded by eight warps from record bytes to bf16 in the same layout,
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
// Roles (640 threads): warp 0 loads dY, warp 1 of the even CTA issues the
// products, warp 2 owns tensor memory, warp 3 reports landed dY tiles to the
// even CTA, warps 4-11 decode, warps 12-19 add up and write.  Two decoder warps
// per scheduler hide each other's shared-memory, conversion and barrier
// latencies.
#include <algorithm>
#include <climits>

#include "taco_host.h"
#include "taco_kernels.h"
#include "taco_tcgen05.cuh"
#include "taco_train.cuh"

namespace taco {
namespace {

__device__ __forceinline__ void store4(float *to, float4 v, int accumulate)
{
    float4 *p = reinterpret_cast<float4 *>(to);
    if (accumulate) {
        const float4 w = *p;
        v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
    }
    *p = v;
}

__device__ __forceinline__ void store4(__nv_bfloat16 *to, float4 v, int accumulate)
{
    uint2 *p = reinterpret_cast<uint2 *>(to);
    if (accumulate) {
        const uint2 w = *p;
        v = make_float4(v.x + __uint_as_float(w.x << 16), v.y + __uint_as_float(w.x & 0xffff0000u),
                        v.z + __uint_as_float(w.y << 16), v.w + __uint_as_float(w.y & 0xffff0000u));
    }
    *p = make_uint2(float2_to_bf16x2(v.x, v.y), float2_to_bf16x2(v.z, v.w));
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
    if (a.dtype == kTypeF32)
        store4(static_cast<float *>(a.dw) + i, v, a.accumulate);
    else
        store4(static_cast<__nv_bfloat16 *>(a.dw) + i, v, a.accumulate);
}

// dW of no rows: four columns a thread.
__global__ void __launch_bounds__(256) taco_weight_grad_empty_kernel(WeightGradArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < a.out * a.hidden; i += 1024ll * gridDim.x) {
        const int64_t m = i / a.hidden;
        finish4(a, m, i - m * a.hidden, a.shift ? a.dy_sum[m] : 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
    }
}

// dY with rows of a multiple of 8 elements: TMA reads rows of whole 16 bytes, so
// where `out` is no multiple of 8 the rows are first copied `width` elements
// apart (zeros behind each), eight elements a thread.
__global__ void __launch_bounds__(256) taco_weight_grad_widen_kernel(const uint16_t *dy, int64_t rows, int64_t out, int64_t width, uint4 *to)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t vectors = width / 8, n = rows * vectors;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += 256ll * gridDim.x) {
        const int64_t r = i / vectors, c = (i - r * vectors) * 8;
        const uint16_t *src = dy + r * out + c;
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 8; k++)
            v[k] = c + k < out ? src[k] : 0u;
        to[i] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
}

// ---------------------------------------------------------------------------
// Tensor-core kernel
// ---------------------------------------------------------------------------

constexpr int kPairM = 256, kPairN = 256;     // tile of a CTA pair; each CTA holds 128 rows of A and of B
constexpr int kStageRows = 64;                // rows of dY and X per pipeline stage
constexpr int kChunkRows = 1024;              // rows per tensor-core accumulation
constexpr int kStages = 4;                    // of both operands and of the record bytes
constexpr int kOperandBytes = 128 * kStageRows * 2;             // one CTA's A or B of a stage
constexpr int kHalfBytes = 64 * kStageRows * 2;                 // 64 columns of it
constexpr int kTeam = 4;                                         // decoder warps of a stage, 16 rows each; two teams
constexpr int kRawWidth = 176;                                   // widest box of record bytes: 4 records of B = 32, and 8 bytes of slack
constexpr int kRawBytes = kStageRows * (kRawWidth + 16);         // even rows, odd rows, then their scales where they lie apart
// Columns that a warp of the epilogue turns round at a time, and its buffer.
constexpr int kTurnColumns = 32, kTurnBytes = 32 * kTurnColumns * 4;
constexpr int kWgThreads = 640;
constexpr size_t kWgSmem = 1024 + static_cast<size_t>(kStages) * 2 * kOperandBytes + kStages * kRawBytes + 8 * kTurnBytes;
constexpr uint32_t kIdesc = mma_idesc_bf16_f32(kPairM, kPairN) | (1u << 15) | (1u << 16);   // A and B MN-major

struct WgBarriers {
    uint64_t a_full[kStages];     // this CTA's dY tile has landed
    uint64_t full[kStages];       // even CTA: both CTAs' A and B of the stage are ready
    uint64_t empty[kStages];      // the stage's products are done
    uint64_t raw_full[kStages];    // record bytes have landed
    uint64_t raw_empty[kStages];   // and have been decoded
    uint64_t acc_full[2];         // a chunk's accumulator is complete
    uint64_t acc_empty[2];        // even CTA: both CTAs have read the accumulator
    uint64_t drained;             // even CTA, after a wait that gave up: the products issued so far are done
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

// An arrival from either CTA.  What it reports lies in the reporting CTA's own
// shared and tensor memory and is read by the tensor core, for which the fences
// before it (fence.proxy.async, tcgen05.fence) order the accesses; a release at
// cluster scope would wait for all of the thread's memory operations besides and
// took 8192 x 16384 x 4096 from 1.95 to 2.78 ms when it was tried.
__device__ __forceinline__ void cluster_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool cluster_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(TACO_WAIT_HINT_NS)
        : "memory");
    return ok != 0;
}

// Bounded wait for a barrier that the other CTA's threads arrive on too.  The
// timer is read only after a first miss: the read alone costs more than a
// stage's products.
__device__ __forceinline__ bool cluster_wait(uint32_t bar, uint32_t parity, uint32_t *fault)
{
    if (cluster_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    while (!cluster_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            atomicOr(fault, kFaultWeightGrad);
            return false;
        }
    }
    return true;
}

// Barrier of the eight epilogue warps: whether `ok` holds for all of them.
__device__ __forceinline__ bool epilogue_agrees(bool ok)
{
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(static_cast<uint32_t>(ok))
        : "memory");
    return all != 0;
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

// The same in this CTA alone, for a barrier that only this thread waits for.
__device__ __forceinline__ void own_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 consecutive tensor-memory columns of this thread's lane, complete on return.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
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

__device__ __forceinline__ float lds_float(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ float4 lds_float4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// Writes a warp's sums, a row of 128 columns a lane: 32 columns at a time go
// through the warp's shared-memory buffer (16-byte units swizzled by the row), so
// that eight lanes then write 128 consecutive bytes of a row.  Written straight
// from the registers, 16 bytes to each of 32 rows an instruction, they kept the
// load/store unit busy for 32 cycles an instruction, which the decoders need too:
// 8192 x 16384 x 4096 took 715 us, turned 686, and 1024^3 16.2 us against 13.0.
// `put(row, col, v)` takes four columns.
template <typename Put>
__device__ __forceinline__ void write_turned(const float (&acc)[128], uint32_t buffer, Put put)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 128; c += kTurnColumns) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kTurnColumns / 4; i++)
            sts128(buffer + lane * 128 + ((i ^ (lane & 7)) << 4),
                   make_uint4(__float_as_uint(acc[c + 4 * i]), __float_as_uint(acc[c + 4 * i + 1]), __float_as_uint(acc[c + 4 * i + 2]),
                              __float_as_uint(acc[c + 4 * i + 3])));
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 32; r += 4) {
            const int row = r + (lane >> 3), unit = lane & 7;
            put(row, c + unit * 4, lds_float4(buffer + row * 128 + ((unit ^ (row & 7)) << 4)));
        }
    }
}

// The grid's work.  Tiles go to the CTA pairs in order (columns fastest); the
// last `tail` tiles, which would leave pairs idle, are cut into `splits` row
// ranges each, whose sums go to `parts` and are joined by a second kernel.
struct WgPlan {
    int64_t units, whole;             // work items, and how many of them are whole tiles
    int tiles_n, stages_total, tail, splits;
    // part: index of the tile's sums in `parts`, or -1 for a whole tile
    __device__ void at(int64_t u, int &m0, int &n0, int64_t &part, int &first, int &count) const
    {
        int64_t t = u;
        first = 0;
        count = stages_total;
        part = -1;
        if (u >= whole) {
            part = u - whole;
            const int split = static_cast<int>(part / tail);
            t = whole + part - static_cast<int64_t>(split) * tail;
            first = static_cast<int>(static_cast<int64_t>(stages_total) * split / splits);
            count = static_cast<int>(static_cast<int64_t>(stages_total) * (split + 1) / splits) - first;
        }
        m0 = static_cast<int>(t / tiles_n) * kPairM;
        n0 = static_cast<int>(t % tiles_n) * kPairN;
    }
};

// Where a CTA's 128 columns from n on lie in a record row, in bytes from the
// start of the row in the map of its parity (see RawMaps).
struct RawSpan {
    int x[2], shift[2];               // box start (16-byte aligned) and first code's offset in the box: even rows, odd rows
    int meta_x[2], meta_shift[2];     // the same for (alpha, s) of blocks above 128
    __device__ RawSpan(int64_t n, int block, int odd_shift)
    {
        const int64_t at = n / block * (block + 8) + n % block, meta = n / block * (block + 8) + block;
#pragma unroll
        for (int p = 0; p < 2; p++) {
            const int64_t c = at + p * odd_shift, m = meta + p * odd_shift;
            x[p] = static_cast<int>(c & ~int64_t{15});
            shift[p] = static_cast<int>(c & 15);
            meta_x[p] = static_cast<int>(m & ~int64_t{15});
            meta_shift[p] = static_cast<int>(m & 15);
        }
    }
};

// Record bytes come by TMA, 64 rows by a CTA's 128 columns at a time.  A record
// row of an odd number of blocks has a length of 8 modulo 16, which no tensor
// map takes as a stride; the rows of each parity lie two lengths apart, so each
// parity has a map of its own.  The odd rows' map then starts 8 bytes before the
// first of them (odd_shift = 8) to be 16-byte aligned.  No map reaches past the
// buffer; rows and columns past the tensor read zeros.  Copying eight bytes a
// lane with cp.async instead took 1.79 ms at 8192 x 16384 x 4096, this 0.84 ms (then).
struct RawMaps {
    CUtensorMap even, odd;            // boxes of `width` bytes by 32 rows
    CUtensorMap meta_even, meta_odd;  // boxes of 16 bytes by 32 rows (blocks above 128)
};

template <int CODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgThreads, 1)
taco_weight_grad_kernel(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ RawMaps raw_maps,
                        WeightGradArgs a, WgPlan plan, int raw_width, int odd_shift, int odd_row0, uint32_t *fault)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) WgBarriers bars;
    __shared__ __align__(16) float affine[512];
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
            mbar_init(bar(bars.full[s]), 2 * (kTeam + 1));   // each CTA's decoders, and its dY tile
            mbar_init(bar(bars.empty[s]), 1);
        }
        for (int s = 0; s < kStages; s++) {
            mbar_init(bar(bars.raw_full[s]), 1);
            mbar_init(bar(bars.raw_empty[s]), kTeam);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(bar(bars.acc_full[b]), 1);
            mbar_init(bar(bars.acc_empty[b]), 16); // eight epilogue warps of each CTA
        }
        mbar_init(bar(bars.drained), 1);
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
            int s = 0;
            uint32_t phase = 0, used = 0;
            bool ok = true;
            for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
                int m0, n0, first, count;
                int64_t part;
                plan.at(u, m0, n0, part, first, count);
                const int x = m0 + static_cast<int>(rank) * 128;
                for (int k = first; k < first + count; k++) {
                    if (!mbar_wait_bounded_thread(bar(bars.empty[s]), phase ^ 1u, fault, kFaultWeightGrad)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = base + s * 2 * kOperandBytes, full = bar(bars.a_full[s]);
                    mbar_arrive_expect_tx(full, kOperandBytes);
                    tma_load_2d(dst, &map_dy, x, k * kStageRows, full);
                    tma_load_2d(dst + kHalfBytes, &map_dy, x + 64, k * kStageRows, full);
                    used |= 1u << s;
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            // No copy may land, and no commit of `empty` from the even CTA arrive, after this CTA is gone: the last phase of
            // every stage that was filled.  That the accumulator's commit was issued after those of `empty` does not order
            // their arrivals.  Once a wait has given up, nothing that is on its way takes as long as that wait did.
            bool arrives = true;
            for (int i = 0; i < kStages; i++)
                if (used >> i & 1u) {
                    const uint32_t last = i < s ? phase : phase ^ 1u;
                    mbar_wait_bounded_thread(bar(bars.a_full[i]), last, fault, kFaultWeightGrad);
                    arrives = arrives && mbar_wait_bounded_thread(bar(bars.empty[i]), last, fault, kFaultWeightGrad);
                }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            int s = 0;
            uint32_t phase = 0, chunk = 0;
            bool ok = true;
            for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
                int m0, n0, first, count;
                int64_t part;
                plan.at(u, m0, n0, part, first, count);
                for (int k = 0; k < count && ok; chunk++) {
                    const int b = static_cast<int>(chunk & 1);
                    if (chunk >= 2 && !cluster_wait(bar(bars.acc_empty[b]), ((chunk >> 1) - 1) & 1u, fault)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const int end = min(count, k + kChunkRows / kStageRows);
                    for (const int begin = k; k < end; k++) {
                        if (!cluster_wait(bar(bars.full[s]), phase, fault)) {
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
                        if (++s == kStages) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
                    if (ok)
                        pair_commit(bar(bars.acc_full[b]));
                }
            }
            if (!ok) {   // no product may read memory that the CTAs give up below
                own_commit(bar(bars.drained));
                mbar_wait_bounded_thread(bar(bars.drained), 0, fault, kFaultWeightGrad);
            }
        } else if (warp == 2 && lane == 0) {
            // Record bytes
            const uint32_t bytes = kStageRows * (raw_width + (a.block > 128 ? 16 : 0));
            int s = 0;
            uint32_t phase = 0, used = 0;
            bool ok = true;
            for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
                int m0, n0, first, count;
                int64_t part;
                plan.at(u, m0, n0, part, first, count);
                const RawSpan at(n0 + static_cast<int64_t>(rank) * 128, a.block, odd_shift);
                for (int k = first; k < first + count; k++) {
                    if (!mbar_wait_bounded_thread(bar(bars.raw_empty[s]), phase ^ 1u, fault, kFaultWeightGrad)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = raw + s * kRawBytes, full = bar(bars.raw_full[s]);
                    const int y = k * (kStageRows / 2);
                    mbar_arrive_expect_tx(full, bytes);
                    tma_load_2d(dst, &raw_maps.even, at.x[0], y, full);
                    tma_load_2d(dst + kStageRows / 2 * kRawWidth, &raw_maps.odd, at.x[1], y + odd_row0, full);
                    if (a.block > 128) {
                        tma_load_2d(dst + kStageRows * kRawWidth, &raw_maps.meta_even, at.meta_x[0], y, full);
                        tma_load_2d(dst + kStageRows * kRawWidth + 512, &raw_maps.meta_odd, at.meta_x[1], y + odd_row0, full);
                    }
                    used |= 1u << s;
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            // no copy may land after the CTA is gone: the last phase of every slot that was filled
            for (int i = 0; i < kStages; i++)
                if (used >> i & 1u)
                    mbar_wait_bounded_thread(bar(bars.raw_full[i]), i < s ? phase : phase ^ 1u, fault, kFaultWeightGrad);
        } else if (warp == 3 && lane == 0) {
            const uint32_t full0 = in_even_cta(bar(bars.full[0]));
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
                int m0, n0, first, count;
                int64_t part;
                plan.at(u, m0, n0, part, first, count);
                for (int k = 0; k < count; k++) {
                    if (!mbar_wait_bounded_thread(bar(bars.a_full[s]), phase, fault, kFaultWeightGrad)) {
                        ok = false;
                        break;
                    }
                    cluster_arrive(full0 + s * 8);
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp < 4 + 2 * kTeam) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // Decoders: two teams of four warps take the stages in turn, so a team's
        // waits, loads and fence run while the other team converts.  Warp d of a
        // team takes rows 16 d .. 16 d + 15 of its stage; lane l the codes 8 (l %
        // 16) .. of rows l / 16, l / 16 + 2, ...
        const int team = (warp - 4) >> 2, d = warp & 3, sub = lane >> 4, col = (lane & 15) * 8;
        const int span = min(a.block, 128);                    // codes of a row's 128 columns lie in pieces of `span`
        const uint32_t swz = static_cast<uint32_t>(lane & 7);
        const uint32_t full0 = in_even_cta(bar(bars.full[0]));
        const uint32_t row_at = static_cast<uint32_t>(sub * (kStageRows / 2) * kRawWidth + d * 8 * raw_width);
        const uint32_t meta_row_at = static_cast<uint32_t>(kStageRows * kRawWidth + sub * 512 + d * 128);
        // Swizzled place of this lane's 16 bytes: row 16 d + 2 j + sub (rows 8 apart share the swizzle).
        uint32_t place[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t kr = static_cast<uint32_t>(2 * j + sub);
            place[j] = static_cast<uint32_t>(kOperandBytes + (col >> 6) * kHalfBytes + d * 2048) + kr * 128 + ((swz ^ kr) << 4);
        }
        int s = 0, turn = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
            int m0, n0, first, count;
            int64_t part;
            plan.at(u, m0, n0, part, first, count);
            const RawSpan at(n0 + static_cast<int64_t>(rank) * 128, a.block, odd_shift);
            const uint32_t code_at = row_at + at.shift[sub] + col / span * (span + 8) + col % span;
            const uint32_t s_at = 4u + (a.block > 128 ? meta_row_at + at.meta_shift[sub]
                                                   : row_at + at.shift[sub] + col / span * (span + 8) + span);
            const uint32_t s_pitch = a.block > 128 ? 16u : static_cast<uint32_t>(raw_width);
            for (int k = 0; k < count; k++, turn ^= 1) {
                if (turn == team) {
                    if (!mbar_wait_bounded(bar(bars.raw_full[s]), phase, fault, kFaultWeightGrad)) {
                        ok = false;
                        break;
                    }
                    const uint32_t src = raw + static_cast<uint32_t>(s) * kRawBytes, dst = base + s * 2 * kOperandBytes;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        uint2 c[4];
                        float f[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            c[j] = lds64(src + code_at + (4 * h + j) * raw_width);
                            f[j] = lds_float(src + s_at + (4 * h + j) * s_pitch);
                        }
                        if (h == 1) {
                            __syncwarp();                      // the warp has read the slot
                            if (lane == 0)
                                mbar_arrive(bar(bars.raw_empty[s]));
                        } else if (!mbar_wait_bounded(bar(bars.empty[s]), phase ^ 1u, fault, kFaultWeightGrad)) {
                            ok = false;
                            break;
                        }
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            sts128(dst + place[j] + h * 1024, decode8<CODE>(c[j], f[j]));
                    }
                    if (!ok)
                        break;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        cluster_arrive(full0 + s * 8);
                }
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        // Epilogue: warp w reads lanes 32 (w % 4) .., columns 128 (w / 4 - 3) .. of the accumulators.
        const int quarter = warp & 3, half = (warp - 12) >> 2;
        const uint32_t empty0 = in_even_cta(bar(bars.acc_empty[0]));
        int64_t chunk = 0;
        bool ok = true;
        for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
            int m0, n0, first, count;
            int64_t part;
            plan.at(u, m0, n0, part, first, count);
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
                for (int c = 0; c < 8; c++) {
                    uint32_t r[16];
                    tmem_ld16(src + c * 16, r);
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        acc[c * 16 + i] += __uint_as_float(r[i]);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    cluster_arrive(empty0 + b * 8);
            }
            // All warps have read the last tile's scales, and go on or give up together (they meet at barriers below).
            ok = epilogue_agrees(ok);
            if (!ok)
                break;
            const int row0 = static_cast<int>(rank) * 128 + quarter * 32;
            const uint32_t buffer = raw + kStages * kRawBytes + (warp - 4 - 2 * kTeam) * kTurnBytes;
            if (part >= 0) {
                float *to = a.parts + (part * kPairM + row0) * kPairN + half * 128;
                write_turned(acc, buffer, [&](int row, int col, float4 v) { *reinterpret_cast<float4 *>(to + row * kPairN + col) = v; });
                continue;
            }
            // scale and shift of the tile's 256 columns as binary32 in shared memory
            const int c = threadIdx.x - (4 + 2 * kTeam) * 32;
            affine[c] = a.scale && n0 + c < a.hidden ? load_param(a.scale, a.param_dtype, n0 + c) : 1.f;
            affine[256 + c] = a.shift && n0 + c < a.hidden ? load_param(a.shift, a.param_dtype, n0 + c) : 0.f;
            named_barrier_sync(1, 256);
            const int64_t mbase = static_cast<int64_t>(m0) + row0, nbase = n0 + half * 128;
            const float own_sum = a.shift && mbase + lane < a.out ? a.dy_sum[mbase + lane] : 0.f;
            write_turned(acc, buffer, [&](int row, int col, float4 v) {
                const float sum = __shfl_sync(kFullMask, own_sum, row);
                if (mbase + row >= a.out || nbase + col >= a.hidden)
                    return;
                const float4 s = *reinterpret_cast<const float4 *>(affine + half * 128 + col);
                const float4 t = *reinterpret_cast<const float4 *>(affine + 256 + half * 128 + col);
                v = make_float4(fmaf(sum, t.x, v.x * s.x), fmaf(sum, t.y, v.y * s.y), fmaf(sum, t.z, v.z * s.z), fmaf(sum, t.w, v.w * s.w));
                const int64_t i = (mbase + row) * a.hidden + nbase + col;
                if (a.dtype == kTypeF32)
                    store4(static_cast<float *>(a.dw) + i, v, a.accumulate);
                else
                    store4(static_cast<__nv_bfloat16 *>(a.dw) + i, v, a.accumulate);
            });
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

// Adds the row ranges' sums of the last tiles in order and finishes four columns a thread.
__global__ void __launch_bounds__(256) taco_weight_grad_join_kernel(WeightGradArgs a, WgPlan plan)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t n = static_cast<int64_t>(plan.tail) * kPairM * kPairN;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < n; i += 1024ll * gridDim.x) {
        const int64_t t = plan.whole + i / (kPairM * kPairN);
        const int64_t m = t / plan.tiles_n * kPairM + i / kPairN % kPairM, col = t % plan.tiles_n * kPairN + i % kPairN;
        if (m >= a.out || col >= a.hidden)
            continue;
        float4 v = *reinterpret_cast<const float4 *>(a.parts + i);
        for (int s = 1; s < plan.splits; s++) {
            const float4 w = *reinterpret_cast<const float4 *>(a.parts + s * n + i);
            v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
        }
        finish4(a, m, col, a.shift ? a.dy_sum[m] : 0.f, v);
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

// Tensor map of [rows, width] elements `pitch` bytes apart, boxes {box_x, box_y}; what lies outside reads zeros.
cudaError_t encode_2d(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t width, int64_t rows, int64_t pitch,
                      int box_x, int box_y, CUtensorMapSwizzle swizzle)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const cudaError_t e = tensor_map_encoder(&encode);
    if (e != cudaSuccess)
        return e;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_y)}, elem_strides[2] = {1, 1};
    return encode(map, type, 2, const_cast<void *>(base), dims, strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t init_weight_grad()
{
    cudaError_t e = cudaSuccess;
    for (int code = 0; code < 3 && e == cudaSuccess; code++)
        e = cudaFuncSetAttribute(wg_kernel(code), cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kWgSmem));
    return e;
}

// Tiles of a weight gradient, how many at the end are cut into row ranges, and
// into how many.  76 pairs take the tiles in waves; what is left for the last
// wave is cut so that all pairs have work, down to 512 rows a range: 8192 x 4096
// x 4096 (256 tiles, 28 of them in the last wave) takes 197 us against 211 whole.
// The pairs of a GB300, not of the current device: the workspace query that shares
// the plan looks at none.  With another count the plan is only less even.
constexpr int64_t kPairs = 76;

struct WgTiles {
    int64_t tiles, tail, splits;
};

WgTiles weight_grad_tiles(int64_t rows, int64_t out, int64_t hidden)
{
    WgTiles w{((out + kPairM - 1) / kPairM) * ((hidden + kPairN - 1) / kPairN), 0, 1};
    w.tail = w.tiles % kPairs;
    if (w.tail > 0)
        w.splits = std::max<int64_t>(1, std::min(kPairs / w.tail, rows / 512));
    if (w.splits == 1)
        w.tail = 0;
    return w;
}

// The row ranges' sums, then dY in rows of a multiple of 8 where it has others.
int64_t weight_grad_part_bytes(const WgTiles &w) { return w.tail * w.splits * kPairM * kPairN * 4; }

int64_t weight_grad_workspace(int64_t rows, int64_t out, int64_t hidden)
{
    return weight_grad_part_bytes(weight_grad_tiles(rows, out, hidden)) + (out % 8 ? 2 * rows * ((out + 7) / 8 * 8) : 0);
}

bool weight_grad_in_range(int64_t rows, int64_t out, int64_t hidden)
{
    // 32-bit TMA coordinates, whole tiles and stages past the end included
    return rows <= INT32_MAX - 64 && out <= INT32_MAX - 256 && hidden <= INT32_MAX / 2;
}

cudaError_t launch_weight_grad(const WeightGradArgs &a, uint32_t *fault, int sms, cudaStream_t stream)
{
    WeightGradArgs args = a;
    if (a.rows == 0) {
        void *p[] = {&args};
        return launch_kernel(reinterpret_cast<void *>(&taco_weight_grad_empty_kernel),
                             static_cast<int>(std::min<int64_t>((a.out * a.hidden + 1023) / 1024, 8ll * sms)), 256, 0, stream, p);
    }
    const WgTiles w = weight_grad_tiles(a.rows, a.out, a.hidden);
    int64_t width = (a.out + 7) / 8 * 8;
    const void *dy = a.dy;
    if (width != a.out) {
        void *to = reinterpret_cast<uint8_t *>(a.parts) + weight_grad_part_bytes(w);
        int64_t rows = a.rows, out = a.out;
        void *p[] = {&dy, &rows, &out, &width, &to};
        const cudaError_t e = launch_kernel(reinterpret_cast<void *>(&taco_weight_grad_widen_kernel),
                                            static_cast<int>(std::min<int64_t>((rows * width + 2047) / 2048, 8ll * sms)), 256, 0,
                                            stream, p);
        if (e != cudaSuccess)
            return e;
        dy = to;
    }
    alignas(64) CUtensorMap map;
    alignas(64) RawMaps raw;
    const int64_t pitch = a.hidden / a.block * (a.block + 8);
    int odd_shift = static_cast<int>(pitch & 8);
    // A row's 128 columns: 128 codes, with (alpha, s) inside up to B = 128, and 8 bytes of slack.
    int raw_width = a.block > 128 ? 144 : (128 / a.block * (a.block + 8) + 8 + 15) / 16 * 16;
    const int64_t even_rows = (a.rows + 1) / 2, odd_rows = a.rows / 2;
    int odd_row0 = odd_rows ? 0 : 1;   // a single row: the odd map holds it too, read from row 1 on, which is outside
    const uint8_t *odd_base = odd_rows ? a.packed + pitch - odd_shift : a.packed;
    cudaError_t e = encode_2d(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, a.out, a.rows, 2 * width, 64, kStageRows,
                              CU_TENSOR_MAP_SWIZZLE_128B);
    for (int i = 0; i < 2 && e == cudaSuccess; i++) {
        const int width = i ? 16 : raw_width;
        e = encode_2d(i ? &raw.meta_even : &raw.even, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.packed, pitch, even_rows, 2 * pitch, width,
                      kStageRows / 2, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (e == cudaSuccess)
            e = encode_2d(i ? &raw.meta_odd : &raw.odd, CU_TENSOR_MAP_DATA_TYPE_UINT8, odd_base, odd_rows ? pitch + odd_shift : pitch,
                          std::max<int64_t>(odd_rows, 1), 2 * pitch, width, kStageRows / 2, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    if (e != cudaSuccess)
        return e;
    WgPlan plan;
    plan.tiles_n = static_cast<int>((a.hidden + kPairN - 1) / kPairN);
    plan.stages_total = static_cast<int>((a.rows + kStageRows - 1) / kStageRows);
    plan.tail = static_cast<int>(w.tail);
    plan.splits = static_cast<int>(w.splits);
    plan.whole = w.tiles - w.tail;
    plan.units = plan.whole + w.tail * w.splits;
    void *p[] = {&map, &raw, &args, &plan, &raw_width, &odd_shift, &odd_row0, &fault};
    e = launch_pairs(wg_kernel(a.code), static_cast<int>(std::min<int64_t>(plan.units, sms / 2)), stream, p);
    if (e == cudaSuccess && plan.tail > 0) {
        void *q[] = {&args, &plan};
        e = launch_kernel(reinterpret_cast<void *>(&taco_weight_grad_join_kernel),
                          static_cast<int>(std::min<int64_t>(w.tail * 64, 8ll * sms)), 256, 0, stream, q);
    }
    return e;
}

}  // namespace taco
