// taco_gelu.cu -- GELU with an 8-bit checkpoint of its input, and its backward
// pass from that checkpoint, for GB300 (sm_103a).
//
// Forward: u = x + bias (binary32), y = u Phi(u) with the normal distribution
// function Phi, or the tanh form y = u/2 (1 + tanh(a (u + b u^3))), a =
// sqrt(2/pi), b = 0.044715; the records of u (taco_train.cuh).
//
// Backward, with u decoded from the records: dx = dy (Phi(u) + u phi(u)), or
// the tanh form's slope; dbias = sum over rows of dx; y again when the next
// weight gradient needs it.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "taco_kernels.h"
#include "taco_train.cuh"

namespace taco {
namespace {

constexpr float kTanhA = 0.7978845608028654f, kTanhB = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f, kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float reciprocal_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// |v|, for positive v at most 30, and a NaN kept.  In the gradient the bound keeps +infinity from meeting the tail's
// zero; -infinity does meet it, as in u Phi(u) = -infinity 0, and comes out as NaN.
__device__ __forceinline__ float bounded_abs(float v)
{
    float r;
    asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(v), "f"(30.f), "f"(-v));
    return r;
}

// Upper tail q = 1 - Phi(a) of the normal distribution for a = |u|, and
// E = exp(-a^2 / 2), which the exponential flushes to zero below 2^-126 (a above
// 13.2).  q = erfc(a / sqrt 2) / 2 equals E t Q(t), t = 1 / (1 + 0.3 a): erfc(z)
// exp(z^2) is smooth and falls like 1/z, so a polynomial in t follows it on the
// whole half line.  Q (degree 7) is a least-squares fit reweighted towards the
// smallest largest relative error on 0 <= a <= 14, 1.7e-7 with the coefficients as
// written.  In binary32 the tail is off by at most 2.5e-7 in absolute terms; its
// relative error grows with the exponent's rounding, which weighs a^2 / 2: measured
// 7e-7 up to a = 4, 3.3e-6 up to 9, 7e-6 up to 13.  One exponential and one
// reciprocal serve Phi and, in the gradient, the density too.
//   gelu(u)  = u Phi(u) = u q for u < 0 and u (1 - q) otherwise, which is max(u, 0) - a q
//   gelu'(u) = Phi(u) + u phi(u) = r for u < 0 and 1 - r otherwise, r = q - a phi(a)
// The value alone takes the first form: 8192 x 16384 bf16 with records 132 us against 134.  The gradient takes the
// second one, whose bounded a it has.
__device__ __forceinline__ float2 normal_tail2(float2 a, float2 &e)
{
    const float2 x = mul2(mul2(a, a), both(-0.5f * kLog2e));
    e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
    const float2 d = fma2(a, both(0.3f), both(1.f));
    const float2 t = make_float2(reciprocal_fast(d.x), reciprocal_fast(d.y));
    float2 q = both(0.03567478060722351f);
    q = fma2(q, t, both(-0.1572030931711197f));
    q = fma2(q, t, both(0.20635348558425903f));
    q = fma2(q, t, both(-0.05368363484740257f));
    q = fma2(q, t, both(0.1285616159439087f));
    q = fma2(q, t, both(0.09991350024938583f));
    q = fma2(q, t, both(0.12075395882129669f));
    q = fma2(q, t, both(0.11962930113077164f));
    return mul2(mul2(q, t), e);
}

// 1 / (1 + exp(-2 v)) = (1 + tanh v) / 2 for v = a (u + b u^3).
__device__ __forceinline__ float2 tanh_gate2(float2 u)
{
    const float2 poly = fma2(mul2(u, u), both(kTanhA * kTanhB), both(kTanhA));
    const float2 x = mul2(mul2(poly, u), both(-2.f * kLog2e));
    return make_float2(reciprocal_fast(1.f + exp2_fast(x.x)), reciprocal_fast(1.f + exp2_fast(x.y)));
}

template <bool TANH>
__device__ __forceinline__ float2 gelu_value2(float2 u)
{
    if (TANH)
        return mul2(u, tanh_gate2(u));
    float2 e;
    const float2 q = normal_tail2(make_float2(fabsf(u.x), fabsf(u.y)), e), p = add2(both(1.f), make_float2(-q.x, -q.y));
    return mul2(u, make_float2(u.x < 0.f ? q.x : p.x, u.y < 0.f ? q.y : p.y));
}

// gelu(u) and its slope.
template <bool TANH>
__device__ __forceinline__ void gelu_both2(float2 u, float2 &y, float2 &slope)
{
    if (TANH) {
        const float2 g = tanh_gate2(u);
        // Beyond |u| = 16 the gate is 0 or 1 and its slope 0; the clamp keeps u^2 finite.
        const float2 c = make_float2(fminf(fmaxf(u.x, -16.f), 16.f), fminf(fmaxf(u.y, -16.f), 16.f));
        const float2 inner = fma2(mul2(c, c), both(6.f * kTanhA * kTanhB), both(2.f * kTanhA));
        const float2 rest = fma2(g, make_float2(-g.x, -g.y), g);          // g (1 - g)
        slope = fma2(mul2(c, inner), rest, g);
        // What is not above -infinity gives NaN, as y = u g does; it does not pass the clamp.  Asked of u: asked of y, 8192 x
        // 16384 takes 169 us against 160.
        if (!(u.x >= -FLT_MAX))
            slope.x = __uint_as_float(0x7fc00000u);
        if (!(u.y >= -FLT_MAX))
            slope.y = __uint_as_float(0x7fc00000u);
        y = mul2(u, g);
    } else {
        float2 e;
        const float2 a = make_float2(bounded_abs(u.x), bounded_abs(u.y)), minus = make_float2(-a.x, -a.y);
        const float2 q = normal_tail2(a, e);
        const float2 r = fma2(mul2(minus, both(kInvSqrt2Pi)), e, q);
        // A choice rather than 1/2 + sign(u) (1/2 - r), in which r below 0 would lose what lies under 3e-8.
        const float2 h = add2(both(1.f), make_float2(-r.x, -r.y));
        slope = make_float2(u.x < 0.f ? r.x : h.x, u.y < 0.f ? r.y : h.y);
        y = fma2(minus, q, make_float2(fmaxf(u.x, 0.f), fmaxf(u.y, 0.f)));
    }
}

// Whole vectors of eight: a warp takes 512 consecutive elements at a time, two
// vectors a lane (the layout of block_max), with the next ones' loads in flight.
// CODE: code format of the records, or -1 for none.
template <typename T, bool TANH, int CODE>
__global__ void __launch_bounds__(256, 4) taco_gelu_kernel(GeluArgs a)
{
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t n = a.rows * a.hidden, step = static_cast<int64_t>(gridDim.x) * 8 * 512;
    int64_t at = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 512 + lane * 8;
    const T *x = static_cast<const T *>(a.x);
    // Column of the first vector, kept up by adding the step modulo the width.
    const int C = static_cast<int>(a.hidden), col_step = static_cast<int>(step % C), col_next = 256 % C;
    int col = static_cast<int>(at % C);
    const int shift = CODE >= 0 ? 31 - __clz(a.block) : 0;
    if (lane == 0 && at < n)   // the warp's first elements on their way to L2 while the kernel before still runs
        bulk_prefetch_l2(x + at, static_cast<uint32_t>((n - at < 512 ? n - at : 512) * sizeof(T)));
    grid_dependency_wait();
    Raw8<T> next[2];
    auto fetch = [&](int64_t i) {
#pragma unroll
        for (int j = 0; j < 2; j++)
            if (i + 256 * j < n)
                next[j] = load_raw8(x + i + 256 * j);
    };
    fetch(at);
    // Every lane of a warp that has work goes round together.
    for (; at - lane * 8 < n; at += step) {
        F8 u[2];
#pragma unroll
        for (int j = 0; j < 2; j++)
            u[j] = unpack(next[j]);
        fetch(at + step);
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                int c = col + j * col_next;
                c = c >= C ? c - C : c;
                const F8 b = load_param_f8(a.bias, a.param_dtype, c);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    u[j].v[i] = add2(u[j].v[i], b.v[i]);
            }
        }
        col += col_step;
        col = col >= C ? col - C : col;
#pragma unroll
        for (int j = 0; j < 2; j++)
            if (at + 256 * j < n) {
                F8 y;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    y.v[i] = gelu_value2<TANH>(u[j].v[i]);
                store_raw8(static_cast<T *>(a.y) + at + 256 * j, pack<T>(y));
            }
        if (CODE >= 0) {
            uint32_t top[2] = {block_max(u[0], a.block), block_max(u[1], a.block)};
            if (a.block == 512)
                top[0] = top[1] = max(top[0], top[1]);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int64_t i = at + 256 * j;
                if (i < n)
                    write_codes<CODE>(u[j], top[j], a.packed + i + (i >> shift) * 8, static_cast<int>(i & (a.block - 1)), a.block);
            }
        }
    }
}

// Widths that are no multiple of 8 (no records then): element by element.
template <typename T>
__global__ void __launch_bounds__(256) taco_gelu_any_kernel(GeluArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t n = a.rows * a.hidden;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += 256ll * gridDim.x) {
        float u = to_float(static_cast<const T *>(a.x)[i]);
        if (a.bias)
            u += load_param(a.bias, a.param_dtype, i % a.hidden);
        const float2 y = a.tanh_form ? gelu_value2<true>(make_float2(u, u)) : gelu_value2<false>(make_float2(u, u));
        static_cast<T *>(a.y)[i] = from_float<T>(y.x);
    }
}

// Gradient: a CTA takes a strip of `strip` vectors of eight columns (at most 32,
// strips of even size), a thread one of them in every 512 / strip-th row, so the
// bias gradient stays in its registers; the CTA's rows are added in order at the
// end.  The next row's loads are in flight.
constexpr int kGradThreads = 512;

template <typename T, bool TANH, int CODE>
__global__ void __launch_bounds__(kGradThreads, 2) taco_gelu_grad_kernel(GeluGradArgs a, int strip)
{
    __shared__ float part[kGradThreads * 8];
    grid_launch_dependents();
    const int rows_a_pass = kGradThreads / strip, mine = threadIdx.x / strip, lane = threadIdx.x - mine * strip;
    const int64_t C = a.hidden, col = (static_cast<int64_t>(blockIdx.x) * strip + lane) * 8;
    const bool in = mine < rows_a_pass && col < C;
    const int64_t step = static_cast<int64_t>(gridDim.y) * rows_a_pass;
    const int64_t block = col / a.block, pitch = C / a.block * (a.block + 8);
    const uint8_t *rec = a.packed + block * (a.block + 8);
    const int within = static_cast<int>(col - block * a.block);
    grid_dependency_wait();
    F8 db;
#pragma unroll
    for (int i = 0; i < 4; i++)
        db.v[i] = both(0.f);
    Raw8<T> next_dy;
    uint2 next_codes = {};
    float next_s = 0.f;
    auto fetch = [&](int64_t row) {
        if (in && row < a.rows) {
            next_dy = load_raw8(static_cast<const T *>(a.dy) + row * C + col);
            next_codes = *reinterpret_cast<const uint2 *>(rec + row * pitch + within);
            next_s = *reinterpret_cast<const float *>(rec + row * pitch + a.block + 4);
        }
    };
    int64_t row = static_cast<int64_t>(blockIdx.y) * rows_a_pass + mine;
    fetch(row);
    if (in)
        for (; row < a.rows; row += step) {
            const F8 g = unpack(next_dy), q = codes8_to_float(next_codes, CODE);
            const float s = next_s;
            fetch(row + step);
            F8 d, y = {};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float2 slope = both(0.f);
                // The second condition always holds.  As a branch it keeps the compiler from interleaving the four pairs of the
                // erf form, which takes 8192 x 16384 bf16 166 us and 8192 x 8192 f32 181; one after the other 162 and 142.
                if (TANH || a.tanh_form == 0)
                    gelu_both2<TANH>(mul2(q.v[i], both(s)), y.v[i], slope);
                d.v[i] = mul2(g.v[i], slope);
                db.v[i] = add2(db.v[i], d.v[i]);
            }
            store_raw8(static_cast<T *>(a.dx) + row * C + col, pack<T>(d));
            if (a.y)
                store_raw8(static_cast<T *>(a.y) + row * C + col, pack<T>(y));
        }
    if (!a.parts)
        return;
    // Sums of the rows that the CTA's threads took, column by column.
#pragma unroll
    for (int i = 0; i < 4; i++) {
        part[2 * i * kGradThreads + threadIdx.x] = db.v[i].x;
        part[(2 * i + 1) * kGradThreads + threadIdx.x] = db.v[i].y;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < strip * 8; c += kGradThreads) {
        const int64_t column = static_cast<int64_t>(blockIdx.x) * strip * 8 + c;
        if (column >= C)
            break;
        float sum = 0.f;
        for (int r = 0; r < rows_a_pass; r++)
            sum += part[(c & 7) * kGradThreads + r * strip + (c >> 3)];
        a.parts[static_cast<int64_t>(blockIdx.y) * C + column] = sum;
    }
}

template <typename T, bool TANH>
const void *gelu_kernel(int code)
{
    return code < 0    ? reinterpret_cast<void *>(&taco_gelu_kernel<T, TANH, -1>)
           : code == 0 ? reinterpret_cast<void *>(&taco_gelu_kernel<T, TANH, 0>)
           : code == 1 ? reinterpret_cast<void *>(&taco_gelu_kernel<T, TANH, 1>)
                       : reinterpret_cast<void *>(&taco_gelu_kernel<T, TANH, 2>);
}

template <typename T, bool TANH>
const void *gelu_grad_kernel(int code)
{
    return code == 0   ? reinterpret_cast<void *>(&taco_gelu_grad_kernel<T, TANH, 0>)
           : code == 1 ? reinterpret_cast<void *>(&taco_gelu_grad_kernel<T, TANH, 1>)
                       : reinterpret_cast<void *>(&taco_gelu_grad_kernel<T, TANH, 2>);
}

template <typename T>
cudaError_t gelu(const GeluArgs &a, int sms, cudaStream_t stream)
{
    GeluArgs args = a;
    void *p[] = {&args};
    const int64_t n = a.rows * a.hidden;
    if (a.hidden % 8 || a.hidden > INT32_MAX / 2) {
        const int64_t want = (n + 255) / 256, cap = static_cast<int64_t>(sms) * 8;
        return launch_kernel(reinterpret_cast<void *>(&taco_gelu_any_kernel<T>), static_cast<int>(std::min(want, cap)), 256, 0, stream, p);
    }
    // Four waves: CTAs that finish early make room (one wave runs 8192 x 16384 with records 6 us longer).
    const int64_t want = (n + 4095) / 4096, cap = static_cast<int64_t>(sms) * 16;
    const int code = a.packed ? a.code : -1;
    return launch_kernel(a.tanh_form ? gelu_kernel<T, true>(code) : gelu_kernel<T, false>(code),
                         static_cast<int>(std::min(want, cap)), 256, 0, stream, p);
}

// Row chunks for a grid of `strips` columns of CTAs: the fewest (up to eight
// waves of the `slots` CTAs that fit the GPU) that leave at most 3% of the slots
// without work, or the best there is.  With 64 strips on 304 slots, 4 chunks
// leave 48 slots idle and 19 fill four waves: 8192 x 16384 takes 164 us
// against 175.
int row_chunks(int64_t strips, int64_t passes, int64_t slots)
{
    const int64_t most = std::min<int64_t>({passes, kMaxColumnParts, std::max<int64_t>(1, 8 * slots / strips)});
    int64_t best = 1;
    double best_share = 0.;
    for (int64_t n = 1; n <= most; n++) {
        const int64_t waves = (strips * n + slots - 1) / slots;
        // the slots' share of work, in whole passes of the longest chunk
        const double share = static_cast<double>(strips * passes) / static_cast<double>(waves * slots * ((passes + n - 1) / n));
        if (share > best_share + 1e-9) {
            best = n;
            best_share = share;
        }
        if (share >= 0.97)
            break;
    }
    return static_cast<int>(best);
}

template <typename T>
cudaError_t gelu_grad(GeluGradArgs *a, int sms, cudaStream_t stream)
{
    const int64_t vectors = a->hidden / 8, strips = (vectors + 31) / 32;
    int strip = static_cast<int>((vectors + strips - 1) / strips);
    const int64_t rows_a_pass = kGradThreads / strip, passes = (a->rows + rows_a_pass - 1) / rows_a_pass;
    a->nparts = row_chunks(strips, passes, 2 * sms);
    void *p[] = {a, &strip};
    return launch_kernel_2d(a->tanh_form ? gelu_grad_kernel<T, true>(a->code) : gelu_grad_kernel<T, false>(a->code),
                            static_cast<unsigned>(strips),
                            static_cast<unsigned>(a->nparts), kGradThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_gelu(int dtype, const GeluArgs &a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? gelu<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? gelu<__half>(a, sms, stream)
                               : gelu<float>(a, sms, stream);
}

cudaError_t launch_gelu_grad(int dtype, GeluGradArgs *a, int sms, cudaStream_t stream)
{
    return dtype == kTypeBf16  ? gelu_grad<__nv_bfloat16>(a, sms, stream)
           : dtype == kTypeF16 ? gelu_grad<__half>(a, sms, stream)
                               : gelu_grad<float>(a, sms, stream);
}

}  // namespace taco
