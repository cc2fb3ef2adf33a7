// taco_train_api.cu -- the C ABI of the training operators (declared in
// include/taco.h): argument validation, workspace layout and launches.
#include <climits>
#include <cmath>
#include <cstdint>

#include "taco.h"
#include "taco_host.h"
#include "taco_train.h"

namespace taco {
namespace {

// A tensor of a call; an absent one (null pointer or no bytes) is skipped.
struct Span {
    const void *p;
    int64_t bytes;
    bool out;
};

// Alignment of every tensor, and no output overlapping another tensor.
template <int N>
taco_status_t check_spans(const Span (&s)[N])
{
    for (const Span &a : s)
        if (!aligned16(a.p))
            return TACO_ERR_MISALIGNED;
    for (int i = 0; i < N; i++)
        for (int j = i + 1; j < N; j++)
            if ((s[i].out || s[j].out) && s[i].p && s[j].p && s[i].bytes && s[j].bytes &&
                overlap(s[i].p, s[i].bytes, s[j].p, s[j].bytes))
                return TACO_ERR_OVERLAP;
    return TACO_OK;
}

bool type_known(int dtype) { return dtype >= TACO_DTYPE_BF16 && dtype <= TACO_DTYPE_F32; }

int64_t type_bytes(int dtype) { return dtype == TACO_DTYPE_F32 ? 4 : 2; }

bool code_known(int code) { return code >= TACO_CODE_E4M3 && code <= TACO_CODE_INT8; }

// rows and hidden non-negative, with four bytes an element (and the records) in range.
taco_status_t check_elements(int64_t rows, int64_t hidden, int64_t *n)
{
    if (rows < 0 || hidden < 0 || (rows != 0 && hidden > INT64_MAX / 16 / rows) || hidden > INT64_MAX / 8192)
        return TACO_ERR_BAD_SHAPE;
    *n = rows * hidden;
    return TACO_OK;
}

taco_status_t check_records(int64_t hidden, int block, int code)
{
    if (!code_known(code))
        return TACO_ERR_BAD_OPTIONS;
    if (!block_supported(block))
        return TACO_ERR_UNSUPPORTED_BLOCK;
    return hidden % block ? TACO_ERR_BAD_SHAPE : TACO_OK;
}

int64_t record_bytes(int64_t n, int block) { return n / block * (block + 8); }

int column_parts(int64_t rows)
{
    return static_cast<int>(rows < kMaxColumnParts ? rows : kMaxColumnParts);
}

// Set-up of the current device and, once, of these operators' kernels.
taco_status_t training_device(DeviceState **out)
{
    const taco_status_t st = device_state(out);
    if (st != TACO_OK)
        return st;
    DeviceState *dev = *out;
    std::call_once(dev->train_once, [dev] {
        cudaError_t e = init_weight_grad();
        if (e == cudaSuccess)
            e = init_norm();
        if (e == cudaSuccess)
            e = init_norm_grad();
        dev->train_error = e;
    });
    return dev->train_error == cudaSuccess ? TACO_OK : cuda_fail(dev->train_error);
}

taco_status_t done(cudaError_t e) { return e == cudaSuccess ? TACO_OK : cuda_fail(e); }

}  // namespace
}  // namespace taco

using namespace taco;

extern "C" {

taco_status_t taco_layernorm(const taco_layernorm_args_t *a, taco_stream_t stream)
{
    if (!a || !type_known(a->dtype) || !type_known(a->param_dtype) || !(a->eps >= 0.f) || !a->residual != !a->summed)
        return TACO_ERR_BAD_OPTIONS;
    int64_t n = 0;
    taco_status_t st = check_elements(a->rows, a->hidden, &n);
    if (st == TACO_OK && a->packed)
        st = check_records(a->hidden, a->block, a->code);
    if (st != TACO_OK || n == 0)
        return st;
    if (!a->x || !a->y || !a->mean || !a->rstd)
        return TACO_ERR_NULL_POINTER;
    const int64_t bytes = n * type_bytes(a->dtype), pbytes = a->hidden * type_bytes(a->param_dtype);
    const Span spans[] = {{a->x, bytes, false},          {a->residual, bytes, false}, {a->weight, pbytes, false},
                          {a->bias, pbytes, false},      {a->y, bytes, true},         {a->summed, bytes, true},
                          {a->mean, 4 * a->rows, true},  {a->rstd, 4 * a->rows, true},
                          {a->packed, a->packed ? record_bytes(n, a->block) : 0, true}};
    if ((st = check_spans(spans)) != TACO_OK)
        return st;
    DeviceState *dev = nullptr;
    if ((st = training_device(&dev)) != TACO_OK)
        return st;
    const NormArgs k{a->x,    a->residual, a->weight, a->bias,   a->y,   a->summed,      a->mean,  a->rstd,
                     static_cast<uint8_t *>(a->packed), a->rows, a->hidden, a->eps, a->param_dtype, a->block, a->code};
    return done(launch_norm(a->dtype, k, dev->sm_count, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t taco_layernorm_backward_workspace(int64_t rows, int64_t hidden)
{
    int64_t n = 0;
    if (check_elements(rows, hidden, &n) != TACO_OK)
        return -1;
    return 2 * 4 * column_parts(rows) * hidden;
}

taco_status_t taco_layernorm_backward(const taco_layernorm_backward_args_t *a, taco_stream_t stream)
{
    if (!a || !type_known(a->dtype) || !type_known(a->param_dtype))
        return TACO_ERR_BAD_OPTIONS;
    int64_t n = 0;
    taco_status_t st = check_elements(a->rows, a->hidden, &n);
    if (st == TACO_OK && !a->x && !a->mean && a->rows != 0)
        st = check_records(a->hidden, a->block, a->code);
    if (st != TACO_OK || a->hidden == 0)
        return st;
    // Only now: of [rows, 0] x is null and mean is not.
    if (a->rows != 0 && !a->x != !a->mean)
        return TACO_ERR_BAD_OPTIONS;
    const bool sums = a->dweight || a->dbias;
    const int parts = column_parts(a->rows);
    const int64_t need = taco_layernorm_backward_workspace(a->rows, a->hidden);
    if (a->rows != 0) {
        if (a->x && a->packed)
            return TACO_ERR_BAD_OPTIONS;
        if (!a->dy || !a->rstd || !a->dx || (!a->x && !a->packed) || (sums && !a->workspace))
            return TACO_ERR_NULL_POINTER;
        if (sums && a->workspace_bytes < need)
            return TACO_ERR_BAD_SHAPE;
    } else if (!sums) {
        return TACO_OK;
    }
    const int64_t bytes = n * type_bytes(a->dtype), pbytes = a->hidden * type_bytes(a->param_dtype);
    const Span spans[] = {{a->dy, bytes, false},
                          {a->x, bytes, false},
                          {a->mean, 4 * a->rows, false},
                          {a->rstd, 4 * a->rows, false},
                          {a->packed, a->packed && a->rows != 0 ? record_bytes(n, a->block) : 0, false},
                          {a->weight, pbytes, false},
                          {a->dsummed, bytes, false},
                          {a->dx, bytes, true},
                          {a->dweight, pbytes, true},
                          {a->dbias, pbytes, true},
                          {sums ? a->workspace : nullptr, need, true}};
    if ((st = check_spans(spans)) != TACO_OK)
        return st;
    DeviceState *dev = nullptr;
    if ((st = training_device(&dev)) != TACO_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    float *ws = sums ? static_cast<float *>(a->workspace) : nullptr;
    NormGradArgs k{a->dy, a->x, a->weight, a->dsummed, a->mean, a->rstd, static_cast<const uint8_t *>(a->packed), a->dx,
                   ws, a->rows, a->hidden, a->param_dtype, a->block, a->code, parts};
    cudaError_t e = cudaSuccess;
    if (a->rows != 0)
        e = launch_norm_grad(a->dtype, &k, dev->sm_count, s);
    if (e == cudaSuccess && sums)
        e = launch_column_sums(ws, k.nparts, a->hidden, a->dweight, a->dbias, a->param_dtype, s);
    return done(e);
}

taco_status_t taco_gelu(const taco_gelu_args_t *a, taco_stream_t stream)
{
    if (!a || !type_known(a->dtype) || !type_known(a->param_dtype) || (a->tanh_form != 0 && a->tanh_form != 1))
        return TACO_ERR_BAD_OPTIONS;
    int64_t n = 0;
    taco_status_t st = check_elements(a->rows, a->hidden, &n);
    if (st == TACO_OK && a->packed)
        st = a->hidden > INT32_MAX / 2 ? TACO_ERR_BAD_SHAPE : check_records(a->hidden, a->block, a->code);   // 32-bit columns
    if (st != TACO_OK || n == 0)
        return st;
    if (!a->x || !a->y)
        return TACO_ERR_NULL_POINTER;
    const int64_t bytes = n * type_bytes(a->dtype);
    const Span spans[] = {{a->x, bytes, false},
                          {a->bias, a->hidden * type_bytes(a->param_dtype), false},
                          {a->y, bytes, true},
                          {a->packed, a->packed ? record_bytes(n, a->block) : 0, true}};
    if ((st = check_spans(spans)) != TACO_OK)
        return st;
    DeviceState *dev = nullptr;
    if ((st = training_device(&dev)) != TACO_OK)
        return st;
    const GeluArgs k{a->x, a->bias, a->y, static_cast<uint8_t *>(a->packed), a->rows, a->hidden,
                     a->param_dtype, a->tanh_form, a->block, a->code};
    return done(launch_gelu(a->dtype, k, dev->sm_count, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t taco_gelu_backward_workspace(int64_t rows, int64_t hidden)
{
    int64_t n = 0;
    if (check_elements(rows, hidden, &n) != TACO_OK)
        return -1;
    return 4 * column_parts(rows) * hidden;
}

taco_status_t taco_gelu_backward(const taco_gelu_backward_args_t *a, taco_stream_t stream)
{
    if (!a || !type_known(a->dtype) || !type_known(a->param_dtype) || (a->tanh_form != 0 && a->tanh_form != 1))
        return TACO_ERR_BAD_OPTIONS;
    int64_t n = 0;
    taco_status_t st = check_elements(a->rows, a->hidden, &n);
    if (st == TACO_OK)
        st = check_records(a->hidden, a->block, a->code);
    if (st != TACO_OK || a->hidden == 0)
        return st;
    const int64_t need = taco_gelu_backward_workspace(a->rows, a->hidden);
    if (a->rows != 0) {
        if (!a->dy || !a->packed || !a->dx || (a->dbias && !a->workspace))
            return TACO_ERR_NULL_POINTER;
        if (a->dbias && a->workspace_bytes < need)
            return TACO_ERR_BAD_SHAPE;
    } else if (!a->dbias) {
        return TACO_OK;
    }
    const int64_t bytes = n * type_bytes(a->dtype);
    const Span spans[] = {{a->dy, bytes, false},
                          {a->packed, record_bytes(n, a->block), false},
                          {a->dx, bytes, true},
                          {a->y, bytes, true},
                          {a->dbias, a->hidden * type_bytes(a->param_dtype), true},
                          {a->dbias ? a->workspace : nullptr, need, true}};
    if ((st = check_spans(spans)) != TACO_OK)
        return st;
    DeviceState *dev = nullptr;
    if ((st = training_device(&dev)) != TACO_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    float *ws = a->dbias ? static_cast<float *>(a->workspace) : nullptr;
    GeluGradArgs k{a->dy, static_cast<const uint8_t *>(a->packed), a->dx, a->y, ws, a->rows, a->hidden,
                   a->tanh_form, a->block, a->code, column_parts(a->rows)};
    cudaError_t e = cudaSuccess;
    if (a->rows != 0)
        e = launch_gelu_grad(a->dtype, &k, dev->sm_count, s);
    if (e == cudaSuccess && a->dbias)
        e = launch_column_sums(ws, k.nparts, a->hidden, a->dbias, nullptr, a->param_dtype, s);
    return done(e);
}

int64_t taco_weight_grad_workspace(int64_t rows, int64_t out, int64_t hidden)
{
    int64_t n = 0;
    if (check_elements(rows, hidden, &n) != TACO_OK || check_elements(rows, out, &n) != TACO_OK ||
        check_elements(out, hidden, &n) != TACO_OK)
        return -1;
    return weight_grad_workspace(rows, out, hidden);
}

taco_status_t taco_weight_grad(const taco_weight_grad_args_t *a, taco_stream_t stream)
{
    if (!a || (a->dtype != TACO_DTYPE_BF16 && a->dtype != TACO_DTYPE_F32) || !type_known(a->param_dtype) ||
        (a->accumulate != 0 && a->accumulate != 1))
        return TACO_ERR_BAD_OPTIONS;
    int64_t nx = 0, ny = 0, nw = 0;
    taco_status_t st = check_elements(a->rows, a->hidden, &nx);
    if (st == TACO_OK)
        st = check_elements(a->rows, a->out, &ny);
    if (st == TACO_OK)
        st = check_elements(a->out, a->hidden, &nw);
    if (st == TACO_OK)
        st = check_records(a->hidden, a->block, a->code);
    if (st == TACO_OK && !weight_grad_in_range(a->rows, a->out, a->hidden))
        st = TACO_ERR_BAD_SHAPE;
    if (st != TACO_OK || nw == 0)
        return st;
    // Only now: shift is null where hidden is 0, dy_sum where out is.
    if (!a->shift != !a->dy_sum)
        return TACO_ERR_BAD_OPTIONS;
    const int64_t need = taco_weight_grad_workspace(a->rows, a->out, a->hidden);
    if (!a->dweight || (a->rows != 0 && (!a->dy || !a->packed)) || (need > 0 && !a->workspace))
        return TACO_ERR_NULL_POINTER;
    if (a->workspace_bytes < need)
        return TACO_ERR_BAD_SHAPE;
    const int64_t pbytes = a->hidden * type_bytes(a->param_dtype);
    const Span spans[] = {{a->dy, 2 * ny, false},
                          {a->packed, record_bytes(nx, a->block), false},
                          {a->dweight, nw * type_bytes(a->dtype), true},
                          {a->scale, pbytes, false},
                          {a->shift, pbytes, false},
                          {a->dy_sum, 4 * a->out, false},
                          {need > 0 ? a->workspace : nullptr, need, true}};
    if ((st = check_spans(spans)) != TACO_OK)
        return st;
    DeviceState *dev = nullptr;
    if ((st = training_device(&dev)) != TACO_OK)
        return st;
    const WeightGradArgs k{a->dy, static_cast<const uint8_t *>(a->packed), a->dweight, a->scale, a->shift, a->dy_sum,
                           static_cast<float *>(a->workspace), a->rows, a->out, a->hidden, a->dtype, a->param_dtype,
                           a->accumulate, a->block, a->code};
    return done(launch_weight_grad(k, dev->fault, dev->sm_count, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
