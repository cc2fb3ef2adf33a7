"""Cases of the training operators around the compressed tensors: the layer norm's forward and backward pass, GELU
and its backward pass from an 8-bit checkpoint, and a linear layer's weight gradient from an 8-bit checkpoint.

A checkpoint is a buffer of DS-only records [codes | alpha = 1 | s] whose scale s is the least power of two with
max|u| <= Qmax s.  `run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once)
or, where `own` is set, through the framework's entry points.  `exact` computes it in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
# Code formats: Qmax as (mantissa, exponent) with Qmax = mantissa * 2^exponent, mantissa in [0.5, 1), and the torch type.
_FORMATS = {"e4m3": (0.875, 9, torch.float8_e4m3fn), "e5m2": (0.875, 16, torch.float8_e5m2), "int8": (0.9921875, 7, torch.int8)}
_BLOCKS = (32, 64, 128, 256, 512)
_EPS = 1e-5


def listed():
    return [
        # The smallest call: one sequence's last tokens through a norm, where the launch counts.
        {"name": "norm_4x4096", "op": "norm", "rows": 4, "hidden": 4096, "dtype": "bf16", "params": "f32",
         "residual": True, "records": False, "block": 128, "code": "e4m3"},
        # The norm behind a tensor-parallel AllReduce of the activation workload: residual add, f32 parameters.
        {"name": "norm_8192x4096", "op": "norm", "rows": 8192, "hidden": 4096, "dtype": "bf16", "params": "f32",
         "residual": True, "records": False, "block": 128, "code": "e4m3"},
        # The same in training with the normalised input kept in 8 bits; a ragged number of tokens.
        {"name": "norm_records_8191x5120", "op": "norm", "rows": 8191, "hidden": 5120, "dtype": "bf16",
         "params": "bf16", "residual": False, "records": True, "block": 128, "code": "e4m3"},
        # Backward pass of the activation workload's norm, with the residual stream's gradient.
        {"name": "norm_grad_8192x4096", "op": "norm_grad", "rows": 8192, "hidden": 4096, "dtype": "bf16",
         "params": "f32", "residual": True, "records": False, "block": 128, "code": "e4m3"},
        # The large tensor's norm from its 8-bit checkpoint.
        {"name": "norm_grad_records_16384x8192", "op": "norm_grad", "rows": 16384, "hidden": 8192, "dtype": "bf16",
         "params": "bf16", "residual": False, "records": True, "block": 128, "code": "e4m3"},
        # An odd width, all in 32 bits: a small model's debugging run.
        {"name": "norm_grad_1000x1111", "op": "norm_grad", "rows": 1000, "hidden": 1111, "dtype": "f32",
         "params": "f32", "residual": False, "records": False, "block": 128, "code": "e4m3"},
        # The activation of an MLP four times as wide as the 4096 model, kept in 8 bits.
        {"name": "gelu_8192x16384", "op": "gelu", "rows": 8192, "hidden": 16384, "dtype": "bf16", "params": "f32",
         "bias": True, "tanh": False, "block": 128, "code": "e4m3"},
        # A short odd batch in f16 with the INT8 fallback and the tanh form.
        {"name": "gelu_333x4096", "op": "gelu", "rows": 333, "hidden": 4096, "dtype": "f16", "params": "f16",
         "bias": True, "tanh": True, "block": 64, "code": "int8"},
        # Its backward pass: the gradient, the bias gradient and the activation again for the next weight gradient.
        {"name": "gelu_grad_8192x16384", "op": "gelu_grad", "rows": 8192, "hidden": 16384, "dtype": "bf16",
         "params": "f32", "bias": True, "tanh": False, "again": True, "block": 128, "code": "e4m3"},
        # A small one with E5M2 codes and the smallest block.
        {"name": "gelu_grad_640x5120", "op": "gelu_grad", "rows": 640, "hidden": 5120, "dtype": "bf16",
         "params": "bf16", "bias": True, "tanh": True, "again": False, "block": 32, "code": "e5m2"},
        # The MLP's first weight gradient (f32) from the norm's checkpoint, with the norm's weight and bias.
        {"name": "weight_grad_8192x16384x4096", "op": "weight_grad", "rows": 8192, "out": 16384, "hidden": 4096,
         "result": "f32", "affine": True, "block": 128, "code": "e4m3"},
        # A small ragged micro-batch into a bf16 gradient.
        {"name": "weight_grad_257x1000x1024", "op": "weight_grad", "rows": 257, "out": 1000, "hidden": 1024,
         "result": "bf16", "affine": False, "block": 32, "code": "int8"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "gelu", "gelu_grad", "weight_grad"))
    block, code = rng.choice(_BLOCKS), rng.choice(tuple(_FORMATS))
    if op == "weight_grad":
        hidden = block * max(1, _spread(rng, 128, 8192) // block)
        out = _spread(rng, 16, 16384)
        out += -out % rng.choice((1, 8, 64, 128))
        rows = _spread(rng, 16, min(16384, max(32, (8192 * 16384 * 4096) // (out * hidden))))
        return {"op": op, "rows": rows, "out": out, "hidden": hidden, "result": rng.choice(("f32", "bf16")),
                "affine": rng.random() < 0.5, "block": block, "code": code}
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    records = op.startswith("gelu") or rng.random() < 0.5
    hidden = _spread(rng, 64, 16384)
    if records:
        hidden = block * max(1, hidden // block)
    elif rng.random() < 0.6:
        hidden = 64 * max(1, hidden // 64)
    rows = _spread(rng, 1, min(16384, (8192 * 8192) // hidden))
    case = {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "params": rng.choice(("f32", dtype)),
            "block": block, "code": code}
    if op.startswith("norm"):
        case.update(residual=rng.random() < 0.5, records=records)
    else:
        case.update(bias=rng.random() < 0.7, tanh=rng.random() < 0.5)
        if op == "gelu_grad":
            case.update(again=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activation(gen, rows, hidden):
    """Channels of very different size, a few outliers and a mean per token, as a residual stream has them."""
    x = _normal(gen, rows, hidden)
    x *= torch.exp(_normal(gen, 1, hidden) * 0.7)
    x *= 1 + 7 * (torch.rand(rows, hidden, generator=gen, device="cuda") < 1e-3)
    return x.add_(0.3 * _normal(gen, rows, 1) + 0.1)


def _gradient(gen, rows, hidden):
    """Small values whose size varies by token; one token in sixteen is padding and has none."""
    g = _normal(gen, rows, hidden)
    size = 1e-2 * torch.exp(_normal(gen, rows, 1) * 0.5)
    return g * size * (torch.rand(rows, 1, generator=gen, device="cuda") >= 1 / 16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, hidden, op = case["rows"], case["hidden"], case["op"]
    state = {"case": case}
    if op == "weight_grad":
        state["dy"] = _gradient(gen, rows, case["out"]).to(torch.bfloat16)
        x = _normal(gen, rows, hidden) * torch.exp(_normal(gen, 1, hidden) * 0.3)
        state["packed"] = _records(x, case["block"], case["code"])
        if case["affine"]:
            state["scale"] = 1 + 0.2 * _normal(gen, hidden)
            state["shift"] = 0.1 * _normal(gen, hidden)
            state["dy_sum"] = state["dy"].float().sum(0)
        return state
    act, param = _DTYPES[case["dtype"]], _DTYPES[case["params"]]
    if op == "norm":
        state["x"] = _activation(gen, rows, hidden).to(act)
        state["weight"] = (1 + 0.2 * _normal(gen, hidden)).to(param)
        state["bias"] = (0.1 * _normal(gen, hidden)).to(param)
        state["residual"] = _activation(gen, rows, hidden).to(act) if case["residual"] else None
    elif op == "norm_grad":
        x = _activation(gen, rows, hidden).to(act)
        state["weight"] = (1 + 0.2 * _normal(gen, hidden)).to(param)
        state["dy"] = _gradient(gen, rows, hidden).to(act)
        state["dsummed"] = _gradient(gen, rows, hidden).to(act) if case["residual"] else None
        mean = x.float().mean(1)
        centred = x.float() - mean[:, None]
        state["rstd"] = torch.rsqrt(centred.square().mean(1) + _EPS)
        if case["records"]:
            state["packed"] = _records(centred * state["rstd"][:, None], case["block"], case["code"])
        else:
            state.update(x=x, mean=mean)
    else:
        x = (1.2 * _activation(gen, rows, hidden)).to(act)
        bias = (0.2 * _normal(gen, hidden)).to(param) if case["bias"] else None
        if op == "gelu":
            state.update(x=x, bias=bias)
        else:
            state["packed"] = _records(x.float() if bias is None else x.float() + bias.float(), case["block"], case["code"])
            state["dy"] = _gradient(gen, rows, hidden).to(act)
    return state


# ---------------------------------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _quantise(u, block, code):
    """Codes and power-of-two scales of the blocks of u (f32): [blocks, block] in the code's type, [blocks, 1] f32."""
    mantissa, exponent, kind = _FORMATS[code]
    u = u.reshape(-1, block)
    m, e = torch.frexp(u.abs().amax(1, keepdim=True))
    e = (e - exponent + (m > mantissa)).clamp(min=-126)
    s = ((e + 127) << 23).to(torch.int32).view(torch.float32)
    v = u / s
    v = torch.round(v) if code == "int8" else v
    return v.to(kind), torch.where(m == 0, torch.zeros_like(s), s)


def _records(u, block, code):
    """The packed buffer of u: for each block its codes, alpha = 1 and s."""
    q, s = _quantise(u, block, code)
    scales = torch.cat([torch.ones_like(s), s], 1).view(torch.uint8)
    return torch.cat([q.view(torch.uint8), scales], 1).reshape(-1)


def _values(packed, rows, hidden, block, code):
    """What a packed buffer stands for, as f32 [rows, hidden]."""
    records = packed.view(-1, block + 8)
    q = records[:, :block].contiguous().view(_FORMATS[code][2]).float()
    s = records[:, block + 4:].contiguous().view(torch.float32)
    return (q * s).view(rows, hidden)


def _normal_cdf(u):
    return 0.5 * (1 + torch.erf(u * math.sqrt(0.5)))


_TANH_A, _TANH_B = math.sqrt(2 / math.pi), 0.044715


def _gelu(u, tanh):
    if tanh:
        return 0.5 * u * (1 + torch.tanh(_TANH_A * (u + _TANH_B * u * u * u)))
    return u * _normal_cdf(u)


def _gelu_slope(u, tanh):
    if tanh:
        t = torch.tanh(_TANH_A * (u + _TANH_B * u * u * u))
        return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * _TANH_A * (1 + 3 * _TANH_B * u * u)
    return _normal_cdf(u) + u * torch.exp(-0.5 * u * u) * (1 / math.sqrt(2 * math.pi))


def _plain(state):
    case = state["case"]
    op, rows, hidden, block, code = case["op"], case["rows"], case["hidden"], case["block"], case["code"]
    if op == "weight_grad":
        x = _values(state["packed"], rows, hidden, block, code)
        dw = state["dy"].float().t() @ x
        if case["affine"]:
            dw = dw * state["scale"] + state["dy_sum"][:, None] * state["shift"]
        return {"dweight": dw.to(_DTYPES[case["result"]])}
    act, param = _DTYPES[case["dtype"]], _DTYPES[case["params"]]
    if op == "norm":
        h = state["x"].float()
        if case["residual"]:
            h = (h + state["residual"].float()).to(act).float()
        mean = h.mean(1)
        centred = h - mean[:, None]
        rstd = torch.rsqrt(centred.square().mean(1) + _EPS)
        xhat = centred * rstd[:, None]
        out = {"y": (xhat * state["weight"].float() + state["bias"].float()).to(act), "mean": mean, "rstd": rstd}
        if case["residual"]:
            out["summed"] = h.to(act)
        if case["records"]:
            q, s = _quantise(xhat, block, code)
            out["values"] = (q.float() * s).to(torch.bfloat16).view(rows, hidden)
        return out
    if op == "norm_grad":
        rstd = state["rstd"][:, None]
        if case["records"]:
            xhat = _values(state["packed"], rows, hidden, block, code)
        else:
            xhat = (state["x"].float() - state["mean"][:, None]) * rstd
        dy = state["dy"].float()
        a = dy * state["weight"].float()
        dx = rstd * (a - a.mean(1, keepdim=True) - xhat * (a * xhat).mean(1, keepdim=True))
        if case["residual"]:
            dx = dx + state["dsummed"].float()
        return {"dx": dx.to(act), "dweight": (dy * xhat).sum(0).to(param), "dbias": dy.sum(0).to(param)}
    if op == "gelu":
        u = state["x"].float()
        if case["bias"]:
            u = u + state["bias"].float()
        q, s = _quantise(u, block, code)
        return {"y": _gelu(u, case["tanh"]).to(act), "values": (q.float() * s).to(torch.bfloat16).view(rows, hidden)}
    u = _values(state["packed"], rows, hidden, block, code)
    dx = state["dy"].float() * _gelu_slope(u, case["tanh"])
    out = {"dx": dx.to(act)}
    if case["bias"]:
        out["dbias"] = dx.sum(0).to(param)
    if case["again"]:
        out["y"] = _gelu(u, case["tanh"]).to(act)
    return out


# ---------------------------------------------------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------------------------------------------------

def _framework(state):
    import fp8_compression_tensor_gb300 as taco

    case = state["case"]
    op, rows, hidden, block, code = case["op"], case["rows"], case["hidden"], case["block"], case["code"]
    if op == "weight_grad":
        dw = taco.weight_grad(state["dy"], state["packed"], hidden, block=block, code=code, scale=state.get("scale"),
                              shift=state.get("shift"), dy_sum=state.get("dy_sum"), dtype=_DTYPES[case["result"]])
        return {"dweight": dw}
    if op == "norm":
        r = taco.layernorm(state["x"], state["weight"], state["bias"], eps=_EPS, residual=state["residual"],
                           checkpoint=case["records"], block=block, code=code)
        out = {"y": r.y, "mean": r.mean, "rstd": r.rstd}
        if case["residual"]:
            out["summed"] = r.summed
        if case["records"]:
            out["values"] = taco.decompress(r.packed, rows, hidden, block=block, variant="ds_only", code=code)
        return out
    if op == "norm_grad":
        g = taco.layernorm_backward(state["dy"], state["rstd"], state["weight"], x=state.get("x"),
                                    mean=state.get("mean"), packed=state.get("packed"), dsummed=state["dsummed"],
                                    block=block, code=code)
        return {"dx": g.dx, "dweight": g.dweight, "dbias": g.dbias}
    approximate = "tanh" if case["tanh"] else "none"
    if op == "gelu":
        r = taco.gelu(state["x"], state["bias"], approximate=approximate, checkpoint=True, block=block, code=code)
        return {"y": r.y, "values": taco.decompress(r.packed, rows, hidden, block=block, variant="ds_only", code=code)}
    g = taco.gelu_backward(state["dy"], state["packed"], approximate=approximate, block=block, code=code,
                           bias_dtype=_DTYPES[case["params"]] if case["bias"] else None, recompute=case["again"])
    out = {"dx": g.dx}
    if case["bias"]:
        out["dbias"] = g.dbias
    if case["again"]:
        out["y"] = g.y
    return out


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    op, rows, hidden, block = case["op"], case["rows"], case["hidden"], case["block"]
    n = rows * hidden
    record = n * (block + 8) / block
    if op == "weight_grad":
        extra = 4 * (2 * hidden + case["out"]) if case["affine"] else 0
        return {"bytes": 2 * rows * case["out"] + record + _BYTES[case["result"]] * case["out"] * hidden + extra,
                "flops": 2 * n * case["out"]}
    e, p = _BYTES[case["dtype"]], _BYTES[case["params"]]
    if op == "norm":
        total = 2 * n * e + 8 * rows + 2 * p * hidden + (2 * n * e if case["residual"] else 0)
        # records are written, read again and returned as bf16 values
        return {"bytes": total + (2 * record + 2 * n if case["records"] else 0), "flops": 8 * n}
    if op == "norm_grad":
        kept = record + 4 * rows if case["records"] else n * e + 8 * rows
        return {"bytes": 2 * n * e + kept + (n * e if case["residual"] else 0) + 3 * p * hidden, "flops": 14 * n}
    params = p * hidden if case["bias"] else 0
    if op == "gelu":
        return {"bytes": 2 * n * e + 2 * record + 2 * n + params, "flops": 16 * n}
    return {"bytes": 2 * n * e + record + (n * e if case["again"] else 0) + params, "flops": 24 * n}


# ---------------------------------------------------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _code_table(code):
    """The value of every code byte, from the formats' definitions."""
    def value(byte):
        if code == "int8":
            return float(byte - 256 if byte > 127 else byte)
        mantissa_bits, bias = (3, 7) if code == "e4m3" else (2, 15)
        e, m = (byte & 127) >> mantissa_bits, byte & ((1 << mantissa_bits) - 1)
        if (code == "e4m3" and byte & 127 == 127) or (code == "e5m2" and e == 31):
            return math.nan if code == "e4m3" or m else math.copysign(math.inf, -1 if byte > 127 else 1)
        size = math.ldexp(m, 1 - bias - mantissa_bits) if e == 0 else math.ldexp(m + (1 << mantissa_bits), e - bias - mantissa_bits)
        return -size if byte > 127 else size
    return torch.tensor([value(b) for b in range(256)], dtype=torch.float64, device="cuda")


def _exact_values(packed, rows, hidden, block, code):
    bytes_ = packed.reshape(-1, block + 8)
    scale = bytes_[:, block + 4:block + 8].contiguous().view(torch.float32).double()
    return (_code_table(code)[bytes_[:, :block].long()] * scale).reshape(rows, hidden)


def _power_of_two(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quantised(u, block, code):
    """u (f64) on the grid of its block: nearest value, ties to the even code."""
    largest, (bits, low) = {"e4m3": (448.0, (3, -6)), "e5m2": (57344.0, (2, -14)), "int8": (127.0, (0, 0))}[code]
    u = u.reshape(-1, block)
    top = u.abs().amax(1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140) / largest)).clamp(min=-126)
    for _ in range(2):   # the least e with top <= largest 2^e, whichever way the logarithm was rounded
        e = torch.where(largest * _power_of_two(e) < top, e + 1, e)
    s = _power_of_two(e)
    v = u / s
    at = torch.zeros_like(v) if code == "int8" else (torch.frexp(v)[1] - 1).clamp(min=low)
    step = _power_of_two(at - bits)
    return torch.round(v / step) * step * s


def _exact_gelu(u, tanh):
    """gelu(u) and its slope."""
    if tanh:
        inner = math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)
        p = torch.sigmoid(2 * inner)
        slope = p + u * 2 * p * torch.sigmoid(-2 * inner) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * u ** 2)
        return u * p, slope
    p = 0.5 * torch.erfc(-u / math.sqrt(2))
    return u * p, p + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    state = prepare(case, seed)
    op, rows, hidden, block, code = case["op"], case["rows"], case["hidden"], case["block"], case["code"]
    if op == "weight_grad":
        x = _exact_values(state["packed"], rows, hidden, block, code)
        if case["affine"]:
            # dY^T (x g + 1 b), with the column sum that the caller holds
            return {"dweight": torch.einsum("rm,rn->mn", state["dy"].double(), x * state["scale"].double())
                    + torch.outer(state["dy_sum"].double(), state["shift"].double())}
        return {"dweight": torch.einsum("rm,rn->mn", state["dy"].double(), x)}
    if op == "norm":
        h = state["x"].double()
        out = {}
        if case["residual"]:
            h = (h + state["residual"].double()).to(_DTYPES[case["dtype"]])
            out["summed"] = h
            h = h.double()
        var, mean = torch.var_mean(h, 1, correction=0)
        rstd = 1 / torch.sqrt(var + _EPS)
        out.update(y=(h - mean[:, None]) * rstd[:, None] * state["weight"].double() + state["bias"].double(), mean=mean, rstd=rstd)
        if case["records"]:
            out["values"] = None   # a normalised value next to a rounding tie takes either code by its 32-bit statistics
        return out
    if op == "norm_grad":
        if case["records"]:
            xhat = _exact_values(state["packed"], rows, hidden, block, code)
        else:
            xhat = (state["x"].double() - state["mean"].double()[:, None]) * state["rstd"].double()[:, None]
        dy = state["dy"].double()
        a = dy * state["weight"].double()
        inner = torch.einsum("rc,rc->r", a, xhat) / hidden
        dx = (a - (a.sum(1) / hidden)[:, None] - xhat * inner[:, None]) * state["rstd"].double()[:, None]
        if case["residual"]:
            dx = dx + state["dsummed"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xhat), "dbias": dy.sum(0)}
    if op == "gelu":
        u = state["x"].double()
        if case["bias"]:
            u = u + state["bias"].double()
        # the records are those of the 32-bit sum u
        return {"y": _exact_gelu(u, case["tanh"])[0], "values": _exact_quantised(u.float().double(), block, code).reshape(rows, hidden)}
    y, slope = _exact_gelu(_exact_values(state["packed"], rows, hidden, block, code), case["tanh"])
    dx = state["dy"].double() * slope
    out = {"dx": dx}
    if case["bias"]:
        out["dbias"] = dx.sum(0)
    if case["again"]:
        out["y"] = y
    return out
