// taco_gated.cu -- gated linear layer (both projections, the activation, the
// product and the 8-bit checkpoint of the projections) and its input's gradient,
// for GB300 (sm_103a).
//
//   z = x W^T + bias,  y = act(z_gate) z_up, records of z;     dx = dz W
//
// A pair of CTAs (a cluster of two) computes a tile of 256 rows with
// tcgen05.mma.cta_group::2 (M = 256, N = 256, K = 16): of the layer 128 columns of
// the gate and the same 128 of the up projection, of dx 256 columns.  Each CTA
// holds 128 rows of A and of B.  For the layer the even CTA loads the gate's rows
// of W and the odd one the up projection's, so one product gives both halves of
// every element to the same thread of the epilogue, and z never leaves the chip
// but as records.  Operands come by TMA (128-byte swizzle; x, W and dz K-major, for
// dx W N-major) in five stages of 64 along K (seven of narrow tiles, 64 columns of
// each projection, where there are few); all copies of a stage count on the
// even CTA's barrier.  Two accumulators of 256 tensor-memory columns take turns, so
// the epilogue of a tile runs beside the next one's products.
//
// Roles (512 threads): warp 0 loads, warp 1 of the even CTA issues the products,
// warp 2 owns tensor memory, warps 4-15 are the epilogue: warp w reads lanes 32 (w
// % 4) .., a row a thread.  Without records the first eight of them take 64 columns
// of y (128 of dx) each; with records the first four take y, the others the gate's
// and the up projection's records.  That took 8192 x 1024 x 4096 with biases from 116
// to 97 us and 333 x 1000 x 2048 f16 with biases from 13.9 to 12.9, against eight
// warps that do both in turn; with what followed they take 92 and (tiles of 64
// columns) 10.1.
//
// One accumulator holds a tile's whole sum.  The tensor core cuts each addition, so
// a sum comes out short by 1.0e-9 of its size a term: measured 8.2e-6 over 8192
// terms, 3.3e-5 over 32768, 1.0e-3 over 2^20, and an eighth of it where a cluster
// cuts the sum (taco_gated_serve.cu).  Outputs have 16 bits, whose rounding alone takes
// 2.1e-4 (f16) or 1.7e-3 (bf16) of one.  The weight gradient, which writes binary32
// and sums over tokens, ends an accumulator after 1024 of them and adds up in
// registers; here that would cost reads and registers for what the outputs' rounding
// hides at the widths of models.
#include <algorithm>
#include <climits>

#include "taco_activation.cuh"
#include "taco_kernels.h"
#include "taco_pair.cuh"

namespace taco {
namespace {

constexpr int kTileM = 256;                   // rows of a pair's tile
constexpr int kStageK = 64;                   // of the sum per pipeline stage
constexpr int kOperandBytes = 128 * kStageK * 2;      // one CTA's A of a stage
constexpr int kHalfBytes = 64 * kStageK * 2;          // 64 columns of an N-major B
constexpr int kThreads = 512;

// Shared memory of a kernel whose tiles have N columns of each projection.
template <int N>
struct Shape {
    static constexpr int kStages = N == 128 ? 5 : 7;
    static constexpr int kStageBytes = kOperandBytes + N * kStageK * 2;   // of one CTA
    // An epilogue warp's buffer for what it writes, and behind it the bias of its columns: without records of one of up to
    // eight warps, with them of four and eight.
    static constexpr int kWarpBytes = N == 128 ? 8192 : 5120, kBiasAt = N == 128 ? 6144 : 4096;
    static constexpr int kOutBytes = 4096 + 1024, kRecordBytes = 40 * N, kRecordWarpBytes = kRecordBytes + 512;
    static constexpr int kBuffers = N == 128 ? 8 * kWarpBytes : 4 * kOutBytes + 8 * kRecordWarpBytes;
    static_assert(4 * kOutBytes + 8 * kRecordWarpBytes <= kBuffers, "buffers");
    static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes + kBuffers;
};
constexpr int kInputGrad = -1;                // in the place of an activation: dx = dz W

template <int kStages>
struct Barriers {
    uint64_t full[kStages];       // even CTA: both CTAs' A and B of the stage have landed
    uint64_t empty[kStages];      // the stage's products are done
    uint64_t acc_full[2];         // an accumulator is complete
    uint64_t acc_empty[2];        // even CTA: both CTAs have read the accumulator
    uint64_t drained;             // even CTA, after a wait that gave up: the products issued so far are done
    uint32_t tmem;
};

// The grid's work.  Tiles go to the CTA pairs in groups of `group_m` row tiles,
// rows fastest, so that the pairs that run at a time share rows of A and of B in
// L2; the last `tail` tiles, which would leave pairs idle, are cut into `splits`
// ranges of K each, whose sums go to `parts` and are joined by a second kernel.
struct Plan {
    int64_t units, whole;             // work items, and how many of them are whole tiles
    int tiles_m, tiles_n, group_m, stages_total, tail, splits;
    __host__ __device__ void tile(int64_t t, int &m, int &n) const
    {
        const int64_t per_group = static_cast<int64_t>(group_m) * tiles_n, g = t / per_group, r = t - g * per_group;
        const int rows = min(group_m, tiles_m - static_cast<int>(g) * group_m);
        m = static_cast<int>(g) * group_m + static_cast<int>(r % rows);
        n = static_cast<int>(r / rows);
    }
    // part: index of the tile's sums in `parts`, or -1 for a whole tile
    __device__ void at(int64_t u, int &m, int &n, int64_t &part, int &first, int &count) const
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
        tile(t, m, n);
    }
};

struct TileArgs {
    void *out;                        // y or dx, [rows, width]
    uint8_t *packed;
    const void *bias;
    float *parts;
    int64_t rows, width;
    int param_dtype, block, code, f16, tma_out;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int f16)
{
    return f16 ? float2_to_f16x2(lo, hi) : float2_to_bf16x2(lo, hi);
}

// A warp's 32 rows of 64 16-bit columns: its buffer holds them in the 128-byte
// swizzle of the output's tensor map.
__device__ __forceinline__ void stage_row32(uint32_t buffer, int lane, int chunk, const float (&v)[32], int f16)
{
#pragma unroll
    for (int i = 0; i < 4; i++)
        sts128(buffer + lane * 128 + (((chunk * 4 + i) ^ (lane & 7)) << 4),
               make_uint4(pack2(v[8 * i], v[8 * i + 1], f16), pack2(v[8 * i + 2], v[8 * i + 3], f16),
                          pack2(v[8 * i + 4], v[8 * i + 5], f16), pack2(v[8 * i + 6], v[8 * i + 7], f16)));
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ float4 lds_float4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// Writes the staged rows to (row, col) of the output: by TMA where its rows are
// whole 16 bytes (what lies outside is not written), otherwise element by element.
__device__ __forceinline__ void write_staged(uint32_t buffer, const void *map, const TileArgs &a, int64_t row, int64_t col)
{
    const int lane = threadIdx.x & 31;
    if (a.tma_out) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row < a.rows && col < a.width) {
            tma_store_2d(map, static_cast<int32_t>(col), static_cast<int32_t>(row), buffer);
            bulk_commit();
        }
        return;
    }
    __syncwarp();
    for (int r = 0; r < 32 && row + r < a.rows; r++)
#pragma unroll
        for (int c = lane; c < 64; c += 32)
            if (col + c < a.width)
                static_cast<uint16_t *>(a.out)[(row + r) * a.width + col + c] =
                    static_cast<uint16_t>(lds16(buffer + r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2));
    __syncwarp();
}

// The bias of a tile's 128 columns from c on, of projection k (0 gate, 1 up), as
// binary32 at `to` in shared memory (zeros outside).  It is fetched ahead of the
// accumulator's wait: loaded a column a lane where it is added, 333 x 1000 x 2048 with
// records (tiles of 128 columns) took 17 us against 13.
__device__ __forceinline__ void stage_bias(uint32_t to, const TileArgs &a, int k, int64_t c)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t col = c + 32 * i + lane;
        const float v = col < a.width ? load_param(a.bias, a.param_dtype, k * a.width + col) : 0.f;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + (32 * i + lane) * 4), "f"(v) : "memory");
    }
}

// 32 accumulators of this thread's row, as loaded, and their columns' staged bias.
__device__ __forceinline__ void to_z(uint32_t (&r)[32], const TileArgs &a, uint32_t bias, float (&z)[32])
{
    tmem_regs_ready(r);
#pragma unroll
    for (int i = 0; i < 32; i++)
        z[i] = __uint_as_float(r[i]);
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 v = lds_float4(bias + i * 4);
            z[i] += v.x;
            z[i + 1] += v.y;
            z[i + 2] += v.z;
            z[i + 3] += v.w;
        }
    }
}

__device__ __forceinline__ void load_z(uint32_t from, const TileArgs &a, uint32_t bias, float (&z)[32])
{
    uint32_t r[32];
    tmem_ld32(from, r);
    tmem_ld_wait();
    to_z(r, a, bias, z);
}

template <int CODE>
__device__ __forceinline__ void encode_row32(const float (&z)[32], float inv, uint32_t to)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float *v = z + 8 * i;
        const uint32_t lo = encode4_scaled(CODE, make_float2(v[0], v[1]), make_float2(v[2], v[3]), inv);
        const uint32_t hi = encode4_scaled(CODE, make_float2(v[4], v[5]), make_float2(v[6], v[7]), inv);
        sts64(to + 8 * i, inv == 0.f ? 0u : lo, inv == 0.f ? 0u : hi);
    }
}

// Records of N columns of one projection (k: 0 gate, 1 up) from column c on, 32
// rows from `row` on; `acc` the first column's accumulators, `bias` its staged bias.
// (N: columns of the tile, 128 or, for blocks up to 64, 64.)
// A block's accumulators are read twice, for its maximum and for its codes.  The
// rows' record bytes go through the buffer (at an odd number of eight bytes apart,
// which the banks like, but for blocks of 32, which fill it) and out in row order.
// The tensor core takes nearly all of shared memory's bandwidth, so what goes
// through the buffers is what an epilogue costs: of 8192 x 1024 x 4096 y takes 4 us
// and the records 14, of 70 without either.  16 bytes a lane on the way out took as
// long.
template <int N>
__device__ __forceinline__ void write_tile_records(uint32_t acc, uint32_t bias, uint32_t buffer, const TileArgs &a, int k, int64_t row,
                                                   int64_t c)
{
    const int lane = threadIdx.x & 31, shift = 31 - __clz(a.block), block = a.block;
    const int cols = static_cast<int>(a.width - c < N ? a.width - c : N);
    const uint32_t pitch = block == 32 ? N + N / 4 : (N / 8 + (N >> shift) | 1) * 8;
    uint32_t to = buffer + lane * pitch;
#pragma unroll 1
    for (int b = 0; b < cols; b += block) {
        uint32_t top = 0;
        float z[32], inv;
#pragma unroll 1
        for (int j = b; j < b + block; j += 32) {
            load_z(acc + j, a, bias + j * 4, z);
#pragma unroll
            for (int i = 0; i < 32; i++)
                top = max(top, abs_bits(z[i]));
        }
        const float s = record_scale(top, a.code, &inv);
#pragma unroll 1
        for (int j = b; j < b + block; j += 32, to += 32) {
            if (block > 32)
                load_z(acc + j, a, bias + j * 4, z);
            if (a.code == 0)
                encode_row32<0>(z, inv, to);
            else if (a.code == 1)
                encode_row32<1>(z, inv, to);
            else
                encode_row32<2>(z, inv, to);
        }
        sts64(to, __float_as_uint(1.f), __float_as_uint(s));
        to += 8;
    }
    __syncwarp();
    const int64_t half = (a.width >> shift) * (block + 8);
    uint8_t *out = a.packed + (row * 2 + k) * half + (c >> shift) * (block + 8);
    const int have = (cols + (cols >> shift) * 8) / 8, rows = static_cast<int>(a.rows - row < 32 ? a.rows - row : 32);
    const int step_r = 32 / have, step_u = 32 - step_r * have;
    int r = lane / have, u = lane - r * have;
    while (r < rows) {
        *reinterpret_cast<uint2 *>(out + r * 2 * half + u * 8) = lds64(buffer + r * pitch + u * 8);
        r += step_r;
        u += step_u;
        if (u >= have) {
            u -= have;
            r++;
        }
    }
    __syncwarp();
}

// N: columns of each projection in a tile (of dx half of its columns).
template <int ACT, int N>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
taco_gated_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_out, TileArgs a, Plan plan, uint32_t idesc, uint32_t *fault)
{
    extern __shared__ uint8_t smem_raw[];
    using S = Shape<N>;
    constexpr int kStages = S::kStages, kStageBytes = S::kStageBytes;
    __shared__ __align__(8) Barriers<kStages> bars;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int64_t first_unit = blockIdx.x >> 1, step_units = gridDim.x >> 1;
    auto bar = [](uint64_t &b) { return smem_addr(&b); };

    grid_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(bar(bars.full[s]), 1);
            mbar_init(bar(bars.empty[s]), 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(bar(bars.acc_full[b]), 1);
            mbar_init(bar(bars.acc_empty[b]), a.packed ? 24 : N == 128 ? 16 : 8);   // the epilogue warps of both CTAs
        }
        mbar_init(bar(bars.drained), 1);
        fence_mbar_init();
        prefetch_tmap(&map_a);
        prefetch_tmap(&map_b);
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

    if (warp == 0 && lane == 0) {
        const uint32_t full0 = in_even_cta(bar(bars.full[0]));
        int s = 0;
        uint32_t phase = 0, used = 0;
        bool ok = true;
        for (int64_t u = first_unit; u < plan.units && ok; u += step_units) {
            int m, n, first, count;
            int64_t part;
            plan.at(u, m, n, part, first, count);
            const int row = m * kTileM + static_cast<int>(rank) * 128;
            for (int k = first; k < first + count; k++) {
                if (!mbar_wait_bounded_thread(bar(bars.empty[s]), phase ^ 1u, fault, kFaultGated)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = base + s * kStageBytes, full = full0 + s * 8;
                if (rank == 0)   // both CTAs' bytes; those of the odd one may have come already
                    mbar_arrive_expect_tx(bar(bars.full[s]), 2 * kStageBytes);
                pair_load_2d(dst, &map_a, k * kStageK, row, full);
                if (ACT == kInputGrad) {
                    const int col = n * 256 + static_cast<int>(rank) * 128;
                    pair_load_2d(dst + kOperandBytes, &map_b, col, k * kStageK, full);
                    pair_load_2d(dst + kOperandBytes + kHalfBytes, &map_b, col + 64, k * kStageK, full);
                } else {
                    pair_load_2d(dst + kOperandBytes, &map_b, k * kStageK, n * N + (rank ? static_cast<int>(a.width) : 0), full);
                }
                used |= 1u << s;
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        // No commit of `empty` may arrive after this CTA is gone, nor a copy land, which the products have waited for: the
        // last phase of every stage that was filled.  Once a wait has given up, nothing that is on its way takes as long as
        // that wait did.
        bool arrives = true;
        for (int i = 0; i < kStages; i++)
            if (used >> i & 1u)
                arrives = arrives && mbar_wait_bounded_thread(bar(bars.empty[i]), i < s ? phase : phase ^ 1u, fault, kFaultGated);
    } else if (warp == 1 && lane == 0 && rank == 0) {
        int s = 0;
        uint32_t phase = 0, turn = 0;
        bool ok = true;
        for (int64_t u = first_unit; u < plan.units && ok; u += step_units, turn++) {
            int m, n, first, count;
            int64_t part;
            plan.at(u, m, n, part, first, count);
            const uint32_t b = turn & 1u;
            if (turn >= 2 && !cluster_wait(bar(bars.acc_empty[b]), ((turn >> 1) - 1) & 1u, fault, kFaultGated)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            for (int k = 0; k < count; k++) {
                if (!cluster_wait(bar(bars.full[s]), phase, fault, kFaultGated)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t sa = base + s * kStageBytes, sb = sa + kOperandBytes;
#pragma unroll
                for (int j = 0; j < kStageK / 16; j++)
                    pair_mma(tmem + b * 256, sw128_kmajor_desc(sa + j * 32),
                             ACT == kInputGrad ? mn_desc(sb + j * 2048, kHalfBytes) : sw128_kmajor_desc(sb + j * 32), idesc, k > 0 || j > 0);
                pair_commit(bar(bars.empty[s]));
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (ok)
                pair_commit(bar(bars.acc_full[b]));
        }
        if (!ok) {   // no product may read memory that the CTAs give up below
            own_commit(bar(bars.drained));
            mbar_wait_bounded_thread(bar(bars.drained), 0, fault, kFaultGated);
        }
    } else if (warp >= 4 && (warp < (N == 128 ? 12 : 8) || a.packed)) {
        const int quarter = warp & 3, team = (warp - 4) >> 2;
        const bool records = ACT != kInputGrad && a.packed;
        const bool out = !records || team == 0;                   // writes y or dx, not records
        const uint32_t empty0 = in_even_cta(bar(bars.acc_empty[0])), buffers = base + kStages * kStageBytes;
        const uint32_t buffer = !records ? buffers + (warp - 4) * S::kWarpBytes
                                : out    ? buffers + quarter * S::kOutBytes
                                         : buffers + 4 * S::kOutBytes + (warp - 8) * S::kRecordWarpBytes;
        const uint32_t bias = buffer + (!records ? S::kBiasAt : out ? 4096 : S::kRecordBytes);
        uint32_t turn = 0;
        for (int64_t u = first_unit; u < plan.units; u += step_units, turn++) {
            int m, n, first, count;
            int64_t part;
            plan.at(u, m, n, part, first, count);
            const uint32_t b = turn & 1u;
            if (ACT != kInputGrad && a.bias) {
                stage_bias(bias, a, out ? 0 : team - 1, static_cast<int64_t>(n) * N);
                if (out)
                    stage_bias(bias + 512, a, 1, static_cast<int64_t>(n) * N);
                __syncwarp();
            }
            if (!mbar_wait_bounded(bar(bars.acc_full[b]), (turn >> 1) & 1u, fault, kFaultGated))
                break;
            tc_fence_after_sync();
            const uint32_t acc = tmem + (static_cast<uint32_t>(quarter) << 21) + b * 256;
            const int row0 = static_cast<int>(rank) * 128 + quarter * 32;
            const int64_t row = static_cast<int64_t>(m) * kTileM + row0;
            if (ACT == kInputGrad && part >= 0) {
                // 32 columns at a time, turned so that eight lanes write 128 consecutive bytes
                float *to = a.parts + (part * kTileM + row0) * 256 + team * 128;
                bulk_wait_read<0>();   // (the lane that stored) the buffer's last tile is on its way
                __syncwarp();
                for (int c = 0; c < 4; c++) {
                    float z[32];
                    load_z(acc + team * 128 + c * 32, a, 0, z);
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        sts128(buffer + lane * 128 + ((i ^ (lane & 7)) << 4),
                               make_uint4(__float_as_uint(z[4 * i]), __float_as_uint(z[4 * i + 1]), __float_as_uint(z[4 * i + 2]),
                                          __float_as_uint(z[4 * i + 3])));
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < 32; r += 4) {
                        const int at = r + (lane >> 3), unit = lane & 7;
                        *reinterpret_cast<float4 *>(to + at * 256 + c * 32 + unit * 4) =
                            lds_float4(buffer + at * 128 + ((unit ^ (at & 7)) << 4));
                    }
                    __syncwarp();
                }
            } else if (ACT == kInputGrad) {
                bulk_wait_read<0>();
                __syncwarp();
                for (int c = 0; c < 2; c++) {
                    const uint32_t place = buffer + c * 4096;
                    for (int j = 0; j < 2; j++) {
                        float z[32];
                        load_z(acc + team * 128 + c * 64 + j * 32, a, 0, z);
                        stage_row32(place, lane, j, z, a.f16);
                    }
                    write_staged(place, &map_out, a, row, static_cast<int64_t>(n) * 256 + team * 128 + c * 64);
                }
            } else if (out) {
                const int64_t c0 = static_cast<int64_t>(n) * N;
                const int begin = records ? 0 : team * 64, end = records ? N : begin + 64;
#pragma unroll 1
                for (int c = begin; c < end; c += 32) {
                    if (c % 64 == 0) {
                        bulk_wait_read<0>();   // (the lane that stored) what the buffer held last is on its way
                        __syncwarp();
                    }
                    uint32_t rg[32], ru[32];
                    tmem_ld32(acc + c, rg);
                    tmem_ld32(acc + N + c, ru);
                    tmem_ld_wait();
                    float g[32], v[32];
                    to_z(rg, a, bias + c * 4, g);
                    to_z(ru, a, bias + 512 + c * 4, v);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 y = mul2(activation2<ACT == kInputGrad ? 0 : ACT>(make_float2(g[i], g[i + 1])), make_float2(v[i], v[i + 1]));
                        v[i] = y.x;
                        v[i + 1] = y.y;
                    }
                    stage_row32(buffer, lane, c >> 5 & 1, v, a.f16);
                    if (c % 64)
                        write_staged(buffer, &map_out, a, row, c0 + c - 32);
                }
            } else {
                write_tile_records<N>(acc + (team - 1) * N, bias, buffer, a, team - 1, row, static_cast<int64_t>(n) * N);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                cluster_arrive(empty0 + b * 8);
        }
        bulk_wait_all<0>();
    }
    tc_fence_before_sync();
    cta_barrier();
    cluster_barrier();
    tc_fence_after_sync();
    __syncwarp();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// The first `joiners` CTAs add the K ranges' sums of the last tiles in order and
// round them, two columns a thread.  The others make column sums (dbias), 32 columns
// a CTA: its eight warps take every eighth part, and the eight sums are added in
// order.  One launch for both: 257 x 1024 x 2752 with dbias 17.4 us, two 20.8.
__global__ void __launch_bounds__(256) taco_gated_join_kernel(TileArgs a, Plan plan, ColumnSums sums, int joiners)
{
    __shared__ float part[8][32];
    grid_launch_dependents();
    grid_dependency_wait();
    if (static_cast<int>(blockIdx.x) >= joiners) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int64_t c = static_cast<int64_t>(blockIdx.x - joiners) * 32 + lane;
        float sum = 0.f;
        if (c < sums.n)
#pragma unroll 4
            for (int i = warp; i < sums.nparts; i += 8)
                sum += sums.parts[i * sums.n + c];
        part[warp][lane] = sum;
        __syncthreads();
        if (warp == 0 && c < sums.n) {
            for (int w = 1; w < 8; w++)
                sum += part[w][lane];
            store_param(sums.out, sums.dtype, c, sum);
        }
        return;
    }
    const int64_t n = static_cast<int64_t>(plan.tail) * kTileM * 256;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 2; i < n; i += 512ll * joiners) {
        int tm, tn;
        plan.tile(plan.whole + i / (kTileM * 256), tm, tn);
        const int64_t row = static_cast<int64_t>(tm) * kTileM + i / 256 % kTileM, col = static_cast<int64_t>(tn) * 256 + i % 256;
        if (row >= a.rows || col >= a.width)
            continue;
        float2 v = *reinterpret_cast<const float2 *>(a.parts + i);
        for (int s = 1; s < plan.splits; s++)
            v = add2(v, *reinterpret_cast<const float2 *>(a.parts + s * n + i));
        const uint32_t w = pack2(v.x, v.y, a.f16);
        uint16_t *to = static_cast<uint16_t *>(a.out) + row * a.width + col;
        to[0] = static_cast<uint16_t>(w);
        if (col + 1 < a.width)
            to[1] = static_cast<uint16_t>(w >> 16);
    }
}

template <int N>
const void *kernel_of(int activation)
{
    return activation == kSilu   ? reinterpret_cast<void *>(&taco_gated_kernel<kSilu, N>)
           : activation == kGelu ? reinterpret_cast<void *>(&taco_gated_kernel<kGelu, N>)
                                 : reinterpret_cast<void *>(&taco_gated_kernel<kGeluTanh, N>);
}

// narrow: 64 columns a tile.
const void *kernel_of(int activation, bool narrow)
{
    return activation == kInputGrad ? reinterpret_cast<void *>(&taco_gated_kernel<kInputGrad, 128>)
           : narrow                 ? kernel_of<64>(activation)
                                    : kernel_of<128>(activation);
}

cudaError_t launch_pairs(const void *fn, size_t smem, int pairs, cudaStream_t stream, void **args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = TACO_PDL ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Row tiles of a group: about 32 MB of A, a quarter of L2, and at least the rows of a square of 76 tiles.
int group_of(int64_t tiles_m, int64_t K)
{
    return static_cast<int>(std::min<int64_t>(tiles_m, std::max<int64_t>(8, (32 << 20) / (kTileM * 2 * K))));
}

int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

// The pairs of a GB300, not of the current device: the workspace query that shares
// the plan of dx looks at none.  With another count the plan is only less even.
constexpr int64_t kPairs = 76;

}  // namespace

cudaError_t init_gated()
{
    cudaError_t e = cudaSuccess;
    for (int act = kInputGrad; act <= kGeluTanh; act++)
        for (int narrow = 0; narrow < (act == kInputGrad ? 1 : 2) && e == cudaSuccess; narrow++)
            e = cudaFuncSetAttribute(kernel_of(act, narrow), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(narrow ? Shape<64>::kSmem : Shape<128>::kSmem));
    return e == cudaSuccess ? init_gated_serve() : e;
}

bool gated_in_range(int64_t rows, int64_t inner, int64_t hidden)
{
    // 32-bit TMA coordinates, whole tiles and stages past the end included
    return rows <= INT32_MAX - 256 && inner <= INT32_MAX / 2 - 256 && hidden <= INT32_MAX - 256;
}

// The epilogue waits for all of a tile's sum at once, for kWaitLimitNs at most.  This many terms take 73 ms at 0.28 us a
// stage of 64, so a launch has time for fourteen times that.
bool gated_sum_in_range(int64_t terms) { return terms <= 1 << 24; }

// x and W in rows of whole 16 bytes where they have others.
int64_t gated_workspace(int64_t rows, int64_t inner, int64_t hidden)
{
    return hidden % 8 ? 2 * (rows + 2 * inner) * up8(hidden) : 0;
}

cudaError_t launch_gated(const GatedArgs &a, uint32_t *fault, int sms, cudaStream_t stream)
{
    const int64_t pitch = up8(a.hidden);
    const void *x = a.x, *w = a.weight;
    cudaError_t e = cudaSuccess;
    if (pitch != a.hidden) {
        uint8_t *ws = static_cast<uint8_t *>(a.workspace);
        e = launch_widen_rows(a.x, a.rows, a.hidden, pitch, ws, sms, stream);
        if (e == cudaSuccess)
            e = launch_widen_rows(a.weight, 2 * a.inner, a.hidden, pitch, ws + 2 * a.rows * pitch, sms, stream);
        x = ws;
        w = ws + 2 * a.rows * pitch;
    }
    if (e == cudaSuccess && !a.packed && gated_serves(a.rows, a.inner))
        return launch_gated_serve(a, x, w, pitch, fault, sms, stream);
    const CUtensorMapDataType type = a.dtype == kTypeF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    alignas(64) CUtensorMap map_x, map_w, map_y = {};
    const bool tma_out = a.inner % 8 == 0;
    // 64 columns a tile where these fit one wave of the pairs, which 128 fill half at most.  A stage then takes 0.23 us (the
    // rate at which an SM's 24 KB come from L2) against 0.28 (its products), in seven stages instead of five, and an
    // epilogue half as long: 256 x 4096 x 3584 20.0 us against 24.4, 512 x 8192 x 2048 34.4 against 41.7.
    const int64_t tiles_m = (a.rows + kTileM - 1) / kTileM;
    const bool narrow = tiles_m * ((a.inner + 63) / 64) <= kPairs && !(a.packed && a.block > 64);
    const int columns = narrow ? 64 : 128;
    if (e == cudaSuccess)
        e = encode_2d(&map_x, type, x, a.hidden, a.rows, 2 * pitch, kStageK, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_2d(&map_w, type, w, a.hidden, 2 * a.inner, 2 * pitch, kStageK, columns, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess && tma_out)
        e = encode_2d(&map_y, type, a.y, a.inner, a.rows, 2 * a.inner, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    Plan plan = {};
    plan.tiles_m = static_cast<int>(tiles_m);
    plan.tiles_n = static_cast<int>((a.inner + columns - 1) / columns);
    plan.group_m = group_of(plan.tiles_m, a.hidden);
    plan.stages_total = static_cast<int>((a.hidden + kStageK - 1) / kStageK);
    plan.whole = plan.units = static_cast<int64_t>(plan.tiles_m) * plan.tiles_n;
    plan.splits = 1;
    TileArgs args{a.y, a.packed, a.bias, nullptr, a.rows, a.inner, a.param_dtype, a.block, a.code, a.dtype == kTypeF16, tma_out};
    uint32_t idesc = a.dtype == kTypeF16 ? mma_idesc_f16_f32(256, 2 * columns) : mma_idesc_bf16_f32(256, 2 * columns);
    void *p[] = {&map_x, &map_w, &map_y, &args, &plan, &idesc, &fault};
    return launch_pairs(kernel_of(a.activation, narrow), narrow ? Shape<64>::kSmem : Shape<128>::kSmem,
                        static_cast<int>(std::min<int64_t>(plan.units, sms / 2)), stream, p);
}

// Tiles of dx, how many at the end are cut into ranges of K, and into how many.
// 76 pairs take the tiles in waves; those of the last wave may be cut so that its
// pairs finish together.  In units of 64 along K (0.27 us a tile) a cut costs what
// its sums take to be written and read again (512 KB a range, 0.2) and the kernel
// that joins them (11): taken where that leaves less than 85%.  With
// the kernel that makes dz, 257 x 1024 x 2752 (8 tiles) takes 15.0 us in the eight
// ranges that this picks (15.2 in seven, 14.6 in nine) and 29.0 whole, 1000 x 2048 x
// 8192 (32 tiles) 65.6 in two and 88.8 whole; 640 x 5120 x 13824 (60 tiles) would
// take 153 cut and takes 143 whole, 8192 x 4096 x 16384 (56 tiles in the last wave
// of 7) 1342 to 1419 either way.
struct Split {
    int64_t tiles, tail, splits;
};

Split input_grad_split(int64_t rows, int64_t inner, int64_t hidden)
{
    const int64_t steps = (2 * inner + kStageK - 1) / kStageK;
    Split s{((rows + kTileM - 1) / kTileM) * ((hidden + 255) / 256), 0, 1};
    s.tail = s.tiles % kPairs;
    int64_t best = 17 * steps;   // twentieths
    for (int64_t n = 2; s.tail > 0 && n <= std::min(std::max<int64_t>(8, kPairs / s.tail), steps / 8); n++) {
        const int64_t time = 20 * ((s.tail * n + kPairs - 1) / kPairs * ((steps + n - 1) / n) + 11) + 4 * s.tail * n;
        if (time < best) {
            best = time;
            s.splits = n;
        }
    }
    if (s.splits == 1)
        s.tail = 0;
    return s;
}

int64_t input_grad_part_bytes(const Split &s) { return s.tail * s.splits * kTileM * 256 * 4; }

// The K ranges' sums, then W in rows of whole 16 bytes where it has others.
int64_t gated_input_grad_workspace(int64_t rows, int64_t inner, int64_t hidden)
{
    return input_grad_part_bytes(input_grad_split(rows, inner, hidden)) + (hidden % 8 ? 4 * inner * up8(hidden) : 0);
}

cudaError_t launch_gated_input_grad(const GatedInputGradArgs &a, const ColumnSums &sums, uint32_t *fault, int sms, cudaStream_t stream)
{
    const Split s = input_grad_split(a.rows, a.inner, a.hidden);
    const int64_t pitch = up8(a.hidden), K = 2 * a.inner;
    const void *w = a.weight;
    cudaError_t e = cudaSuccess;
    if (pitch != a.hidden) {
        void *to = static_cast<uint8_t *>(a.workspace) + input_grad_part_bytes(s);
        e = launch_widen_rows(a.weight, K, a.hidden, pitch, to, sms, stream);
        w = to;
    }
    const CUtensorMapDataType type = a.dtype == kTypeF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    alignas(64) CUtensorMap map_dz, map_w, map_dx = {};
    const bool tma_out = a.hidden % 8 == 0;
    if (e == cudaSuccess)
        e = encode_2d(&map_dz, type, a.dz, K, a.rows, 2 * K, kStageK, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_2d(&map_w, type, w, a.hidden, K, 2 * pitch, 64, kStageK, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess && tma_out)
        e = encode_2d(&map_dx, type, a.dx, a.hidden, a.rows, 2 * a.hidden, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    Plan plan = {};
    plan.tiles_m = static_cast<int>((a.rows + kTileM - 1) / kTileM);
    plan.tiles_n = static_cast<int>((a.hidden + 255) / 256);
    plan.group_m = group_of(plan.tiles_m, K);
    plan.stages_total = static_cast<int>((K + kStageK - 1) / kStageK);
    plan.tail = static_cast<int>(s.tail);
    plan.splits = static_cast<int>(s.splits);
    plan.whole = s.tiles - s.tail;
    plan.units = plan.whole + s.tail * s.splits;
    TileArgs args{a.dx, nullptr, nullptr, static_cast<float *>(a.workspace), a.rows, a.hidden, 0, 0, 0, a.dtype == kTypeF16, tma_out};
    uint32_t idesc = (a.dtype == kTypeF16 ? mma_idesc_f16_f32(256, 256) : mma_idesc_bf16_f32(256, 256)) | (1u << 16);   // B N-major
    void *p[] = {&map_dz, &map_w, &map_dx, &args, &plan, &idesc, &fault};
    e = launch_pairs(kernel_of(kInputGrad, false), Shape<128>::kSmem, static_cast<int>(std::min<int64_t>(plan.units, sms / 2)),
                     stream, p);
    if (e != cudaSuccess)
        return e;
    if (plan.tail > 0) {
        int joiners = static_cast<int>(std::min<int64_t>(s.tail * 128, 8ll * sms));
        ColumnSums columns = sums;
        void *q[] = {&args, &plan, &columns, &joiners};
        const int64_t ctas = joiners + (sums.parts ? (sums.n + 31) / 32 : 0);
        return launch_kernel(reinterpret_cast<void *>(&taco_gated_join_kernel), static_cast<int>(ctas), 256, 0, stream, q);
    }
    return sums.parts ? launch_column_sums(sums.parts, sums.nparts, sums.n, sums.out, nullptr, sums.dtype, stream) : cudaSuccess;
}

}  // namespace taco
