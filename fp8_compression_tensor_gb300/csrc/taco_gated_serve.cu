// taco_gated_serve.cu -- gated linear layer of few rows (the tokens of a decoding
// step), for GB300 (sm_103a).
//
//   z = x W^T + bias,  y = act(z_gate) z_up
//
// With few rows the weights are all that counts: each of them is read once and
// meets `rows` values.  So the operands change places: 64 rows of the gate and the
// same 64 of the up projection are the M = 128 side of tcgen05.mma and the tokens,
// filled up to a multiple of 16, the N side.  A CTA streams its 128 rows of W by
// TMA (128-byte swizzle) through as many stages as fit two CTAs an SM; where the
// inner width gives too few CTAs to fill the GPU, a cluster cuts K and adds its
// CTAs' sums through distributed shared memory, in the order of the CTAs.
#include <algorithm>

#include "taco_activation.cuh"
#include "taco_kernels.h"
#include "taco_pair.cuh"

namespace taco {
namespace {

constexpr int kStageK = 64, kTile = 64, kMaxTokens = 128, kMaxStages = 12, kMaxSplits = 8, kThreads = 128;
constexpr int kWeightBytes = 2 * kTile * kStageK * 2;   // of a stage: gate, up
constexpr size_t kSmemBudget = 113 * 1024;              // two CTAs an SM

struct ServeArgs {
    void *y;
    const void *bias;
    int64_t rows, inner;
    int param_dtype, f16, tokens, stages, stages_total, splits;
};

struct Barriers {
    uint64_t full[kMaxStages];    // the stage has landed
    uint64_t empty[kMaxStages];   // its products are done
    uint64_t done;                // all products are
    uint32_t tmem;
};

// Two floats of shared memory of the cluster's CTA `rank`, at this CTA's address `addr`.
__device__ __forceinline__ float2 peer_float2(uint32_t addr, uint32_t rank)
{
    float2 v;
    asm volatile("{\n\t.reg .u32 p;\n\tmapa.shared::cluster.u32 p, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [p];\n\t}"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

template <int ACT>
__global__ void __launch_bounds__(kThreads)
taco_gated_serve_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, ServeArgs a,
                        uint32_t idesc, uint32_t *fault)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Barriers bars;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = a.splits > 1 ? cluster_rank() : 0u;
    const int n0 = static_cast<int>(blockIdx.x / a.splits) * kTile;
    const int first = a.stages_total * static_cast<int>(rank) / a.splits;
    const int count = a.stages_total * static_cast<int>(rank + 1) / a.splits - first;
    const uint32_t stage_bytes = kWeightBytes + a.tokens * kStageK * 2;
    auto bar = [](uint64_t &b) { return smem_addr(&b); };

    grid_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; s++) {
            mbar_init(bar(bars.full[s]), 1);
            mbar_init(bar(bars.empty[s]), 1);
        }
        mbar_init(bar(bars.done), 1);
        fence_mbar_init();
        prefetch_tmap(&map_x);
        // the first weights on their way to L2 while the kernel before still runs
        for (int k = first; k < first + min(count, a.stages); k++) {
            tma_prefetch_2d(&map_w, k * kStageK, n0);
            tma_prefetch_2d(&map_w, k * kStageK, static_cast<int>(a.inner) + n0);
        }
    }
    if (warp == 2) {
        tmem_alloc(smem_addr(&bars.tmem), kMaxTokens);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    cta_barrier();
    tc_fence_after_sync();
    const uint32_t tmem = bars.tmem;
    grid_dependency_wait();

    if (warp == 0 && lane == 0) {
        int s = 0;
        uint32_t phase = 0, used = 0;
        for (int k = first; k < first + count; k++) {
            if (!mbar_wait_bounded_thread(bar(bars.empty[s]), phase ^ 1u, fault, kFaultGated))
                break;
            const uint32_t dst = base + s * stage_bytes, full = bar(bars.full[s]);
            mbar_arrive_expect_tx(full, stage_bytes);
            tma_load_2d(dst, &map_w, k * kStageK, n0, full);
            tma_load_2d(dst + kWeightBytes / 2, &map_w, k * kStageK, static_cast<int>(a.inner) + n0, full);
            tma_load_2d(dst + kWeightBytes, &map_x, k * kStageK, 0, full);
            used |= 1u << s;
            if (++s == a.stages) {
                s = 0;
                phase ^= 1u;
            }
        }
        // no copy may land and no commit arrive after this CTA is gone: the last phase of every stage that was filled
        bool arrives = true;
        for (int i = 0; i < a.stages; i++)
            if (used >> i & 1u)
                arrives = arrives && mbar_wait_bounded_thread(bar(bars.empty[i]), i < s ? phase : phase ^ 1u, fault, kFaultGated);
    } else if (warp == 1 && lane == 0) {
        int s = 0;
        uint32_t phase = 0;
        for (int k = 0; k < count; k++) {
            if (!mbar_wait_bounded_thread(bar(bars.full[s]), phase, fault, kFaultGated))
                break;
            tc_fence_after_sync();
            const uint32_t sw = base + s * stage_bytes;
#pragma unroll
            for (int j = 0; j < kStageK / 16; j++)
                tc_mma_bf16(tmem, sw128_kmajor_desc(sw + j * 32), sw128_kmajor_desc(sw + kWeightBytes + j * 32), idesc, k > 0 || j > 0);
            tc_commit(bar(bars.empty[s]));
            if (++s == a.stages) {
                s = 0;
                phase ^= 1u;
            }
        }
        tc_commit(bar(bars.done));   // after a wait that gave up too: no product may read memory that is given up below
    }
    __syncwarp();
    const bool ok = mbar_wait_bounded(bar(bars.done), 0, fault, kFaultGated);
    tc_fence_after_sync();
    // Sums [token][128 rows of W] in the stages' place
    if (ok)
        for (int c = 0; c < a.tokens; c += 16) {
            uint32_t r[16];
            tmem_ld16(tmem + (static_cast<uint32_t>(warp) << 21) + c, r);
#pragma unroll
            for (int i = 0; i < 16; i++)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + static_cast<uint32_t>(((c + i) * 128 + threadIdx.x) * 4)), "r"(r[i])
                             : "memory");
        }
    tc_fence_before_sync();
    cta_barrier();
    if (a.splits > 1)
        cluster_barrier();
    if (warp == 2) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kMaxTokens);
    }
    // The cluster's CTAs share out the tokens: two columns a thread
    for (int64_t t = static_cast<int64_t>(rank) * 4 + warp; t < a.rows; t += 4ll * a.splits) {
        const int64_t c = n0 + 2 * lane;
        const uint32_t at = base + static_cast<uint32_t>((t * 128 + 2 * lane) * 4);
        // all CTAs' sums on their way before the first is added
        float2 gate[kMaxSplits], up[kMaxSplits];
#pragma unroll
        for (int p = 0; p < kMaxSplits; p++)
            if (p < a.splits) {
                gate[p] = peer_float2(at, p);
                up[p] = peer_float2(at + 256, p);
            }
        float2 g = gate[0], u = up[0];
#pragma unroll
        for (int p = 1; p < kMaxSplits; p++)
            if (p < a.splits) {
                g = add2(g, gate[p]);
                u = add2(u, up[p]);
            }
        if (c >= a.inner)
            continue;
        const bool second = c + 1 < a.inner;
        if (a.bias) {
            g.x += load_param(a.bias, a.param_dtype, c);
            u.x += load_param(a.bias, a.param_dtype, a.inner + c);
            if (second) {
                g.y += load_param(a.bias, a.param_dtype, c + 1);
                u.y += load_param(a.bias, a.param_dtype, a.inner + c + 1);
            }
        }
        const float2 y = mul2(activation2<ACT>(g), u);
        const uint32_t w = a.f16 ? float2_to_f16x2(y.x, y.y) : float2_to_bf16x2(y.x, y.y);
        uint16_t *to = static_cast<uint16_t *>(a.y) + t * a.inner + c;
        if (a.inner % 2 == 0) {
            *reinterpret_cast<uint32_t *>(to) = w;
        } else {
            to[0] = static_cast<uint16_t>(w);
            if (second)
                to[1] = static_cast<uint16_t>(w >> 16);
        }
    }
    if (a.splits > 1)
        cluster_barrier();   // the other CTAs may still read this one's sums
}

const void *kernel_of(int activation)
{
    return activation == kSilu   ? reinterpret_cast<void *>(&taco_gated_serve_kernel<kSilu>)
           : activation == kGelu ? reinterpret_cast<void *>(&taco_gated_serve_kernel<kGelu>)
                                 : reinterpret_cast<void *>(&taco_gated_serve_kernel<kGeluTanh>);
}

}  // namespace

cudaError_t init_gated_serve()
{
    cudaError_t e = cudaSuccess;
    for (int act = kSilu; act <= kGeluTanh && e == cudaSuccess; act++)
        e = cudaFuncSetAttribute(kernel_of(act), cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBudget));
    return e;
}

// Up to 64 rows always (16384 x 4096 weights: 64 rows 47 us, the pairs' kernel 52);
// up to 128 where the pairs' kernel, whose tiles are 128 columns wide, has no more
// than a wave and a bit of them: 128 rows, 4096 x 2048 13 us against 23, x 12288 46
// against 50, but x 16384 55 against 53.
bool gated_serves(int64_t rows, int64_t inner) { return rows <= 64 || (rows <= kMaxTokens && inner <= 96 * 128); }

cudaError_t launch_gated_serve(const GatedArgs &a, const void *x, const void *w, int64_t pitch, uint32_t *fault, int sms, cudaStream_t stream)
{
    ServeArgs args{a.y, a.bias, a.rows, a.inner, a.param_dtype, a.dtype == kTypeF16, static_cast<int>((a.rows + 15) / 16 * 16),
                   0, static_cast<int>((a.hidden + kStageK - 1) / kStageK), 1};
    const int stage_bytes = kWeightBytes + args.tokens * kStageK * 2;
    const int64_t tiles = (a.inner + kTile - 1) / kTile;
    // Nine tenths of the places: a cluster lies in one processing cluster of SMs, which odd numbers of CTAs do not fill (41
    // tiles of 7 CTAs ran in two waves, 2552 x 2592 in 18.3 us).
    args.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kMaxSplits, 9 * sms / 5 / tiles, args.stages_total / 4})));
    args.stages = std::max(2, std::min({kMaxStages, static_cast<int>((kSmemBudget - 1280) / stage_bytes),
                                        (args.stages_total + args.splits - 1) / args.splits}));
    const CUtensorMapDataType type = args.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    alignas(64) CUtensorMap map_w, map_x;
    cudaError_t e = encode_2d(&map_w, type, w, a.hidden, 2 * a.inner, 2 * pitch, kStageK, kTile, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_2d(&map_x, type, x, a.hidden, a.rows, 2 * pitch, kStageK, args.tokens, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    uint32_t idesc = args.f16 ? mma_idesc_f16_f32(128, args.tokens) : mma_idesc_bf16_f32(128, args.tokens);
    void *p[] = {&map_w, &map_x, &args, &idesc, &fault};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * args.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + static_cast<size_t>(args.stages) * stage_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(args.splits);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = TACO_PDL ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, kernel_of(a.activation), p);
}

}  // namespace taco
