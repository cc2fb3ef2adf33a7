"""Cases of the operators of a gated feed-forward block behind a root-mean-square norm: the norm with the residual's
addition and 8-bit outputs, its gradient, the gated linear layer (both projections, the activation and the product)
with an 8-bit checkpoint, and its gradient from that checkpoint.

8-bit values are buffers of DS-only records [codes | alpha = 1 | s] whose scale s is the least power of two with
max|u| <= Qmax s.  `run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once) or,
where `own` is set, through the framework's entry points.  `exact` computes it in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
# Code formats: Qmax as (mantissa, exponent) with Qmax = mantissa * 2^exponent, mantissa in [0.5, 1), and the torch type.
_FORMATS = {"e4m3": (0.875, 9, torch.float8_e4m3fn), "e5m2": (0.875, 16, torch.float8_e5m2), "int8": (0.9921875, 7, torch.int8)}
_BLOCKS = (32, 64, 128, 256, 512)
_GATED_BLOCKS = (32, 64, 128)
_ACTIVATIONS = ("silu", "gelu", "gelu_tanh")
_EPS = 1e-6


def _norm_case(name, rows, hidden, dtype, params, residual, checkpoint, packed_y, block=128, code="e4m3"):
    return {"name": name, "op": "norm", "rows": rows, "hidden": hidden, "dtype": dtype, "params": params,
            "residual": residual, "checkpoint": checkpoint, "packed_y": packed_y, "block": block, "code": code}


def _norm_grad_case(name, rows, hidden, dtype, params, residual, records, block=128, code="e4m3"):
    return {"name": name, "op": "norm_grad", "rows": rows, "hidden": hidden, "dtype": dtype, "params": params,
            "residual": residual, "records": records, "block": block, "code": code}


def _gated_case(name, rows, hidden, inner, dtype, activation, bias, checkpoint, block=128, code="e4m3"):
    return {"name": name, "op": "gated", "rows": rows, "hidden": hidden, "inner": inner, "dtype": dtype,
            "activation": activation, "bias": bias, "checkpoint": checkpoint, "block": block, "code": code}


def _gated_grad_case(name, rows, hidden, inner, dtype, activation, bias, again, block=128, code="e4m3"):
    return {"name": name, "op": "gated_grad", "rows": rows, "hidden": hidden, "inner": inner, "dtype": dtype,
            "activation": activation, "bias": bias, "again": again, "block": block, "code": code}


def listed():
    return [
        # The smallest call: the last tokens of four sequences through a norm, where the launch counts.
        _norm_case("rms_4x4096", 4, 4096, "bf16", "bf16", True, False, False),
        # The norm behind a tensor-parallel AllReduce of the activation workload, its output in 8 bits to be gathered
        # by the other ranks, and the normalised rows kept in 8 bits for the backward pass.
        _norm_case("rms_packed_8192x4096", 8192, 4096, "bf16", "f32", True, True, True),
        # A ragged number of tokens at an odd width, all in 32 bits.
        _norm_case("rms_1023x2055", 1023, 2055, "f32", "f32", False, False, False),
        # Backward pass of the activation workload's norm, with the residual stream's gradient.
        _norm_grad_case("rms_grad_8192x4096", 8192, 4096, "bf16", "f32", True, False),
        # The large tensor's norm from its 8-bit checkpoint.
        _norm_grad_case("rms_grad_records_16384x8192", 16384, 8192, "bf16", "bf16", False, True),
        # One token through the gated layer of a 4096 model: the weights are read for it alone.
        _gated_case("gated_1x4096x16384", 1, 4096, 16384, "bf16", "silu", False, False),
        # A batch of 48 sequences, a token each, through a rank's share of the 5120 model's gated layer.
        _gated_case("gated_48x5120x3456", 48, 5120, 3456, "bf16", "silu", False, False),
        # The training step's forward pass at the activation workload's size, kept in 8 bits.
        _gated_case("gated_records_8192x4096x16384", 8192, 4096, 16384, "bf16", "silu", False, True),
        # A short ragged batch in f16, with biases, the tanh form and INT8 codes.
        _gated_case("gated_333x1000x2048", 333, 1000, 2048, "f16", "gelu_tanh", True, True, 64, "int8"),
        # The training step's backward pass: both projections' gradients, the input's, and the product again for the
        # down projection's weight gradient.
        _gated_grad_case("gated_grad_8192x4096x16384", 8192, 4096, 16384, "bf16", "silu", False, True),
        # A small ragged micro-batch with bias gradients, the erf form, the smallest block and E5M2 codes.
        _gated_grad_case("gated_grad_257x1024x2752", 257, 1024, 2752, "bf16", "gelu", True, False, 32, "e5m2"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "gated", "gated", "gated_grad"))
    code = rng.choice(tuple(_FORMATS))
    if op.startswith("gated"):
        block = rng.choice(_GATED_BLOCKS)
        records = op == "gated_grad" or rng.random() < 0.5
        hidden = _spread(rng, 64, 8192)
        if rng.random() < 0.85:
            hidden = 8 * (hidden // 8)
        inner = _spread(rng, 32, 16384)
        if records:
            inner = block * max(1, inner // block)
        elif rng.random() < 0.8:
            inner = 8 * (inner // 8)
        rows = _spread(rng, 1, min(8192, max(2, (8192 * 4096 * 16384) // (hidden * inner))))
        case = {"op": op, "rows": rows, "hidden": hidden, "inner": inner, "dtype": rng.choice(("bf16", "bf16", "f16")),
                "activation": rng.choice(_ACTIVATIONS), "bias": rng.random() < 0.3, "block": block, "code": code}
        case["again" if op == "gated_grad" else "checkpoint"] = records if op == "gated" else rng.random() < 0.5
        return case
    block = rng.choice(_BLOCKS)
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    hidden = _spread(rng, 64, 16384)
    first, second = rng.random() < 0.5, rng.random() < 0.3
    if first or (op == "norm" and second):
        hidden = block * max(1, hidden // block)
    elif rng.random() < 0.6:
        hidden = 64 * max(1, hidden // 64)
    rows = _spread(rng, 1, min(16384, (8192 * 8192) // hidden))
    case = {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "params": rng.choice(("f32", dtype)),
            "residual": rng.random() < 0.5, "block": block, "code": code}
    case.update({"checkpoint": first, "packed_y": second} if op == "norm" else {"records": first})
    return case


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activation_rows(gen, rows, hidden):
    """Channels of very different size and a few outliers, as a residual stream has them."""
    x = _normal(gen, rows, hidden)
    x *= torch.exp(_normal(gen, 1, hidden) * 0.7)
    x *= 1 + 7 * (torch.rand(rows, hidden, generator=gen, device="cuda") < 1e-3)
    return x


def _gradient(gen, rows, hidden):
    """Small values whose size varies by token; one token in sixteen is padding and has none."""
    g = _normal(gen, rows, hidden)
    size = 1e-2 * torch.exp(_normal(gen, rows, 1) * 0.5)
    return g * size * (torch.rand(rows, 1, generator=gen, device="cuda") >= 1 / 16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, hidden, op, act = case["rows"], case["hidden"], case["op"], _DTYPES[case["dtype"]]
    state = {"case": case}
    if op == "norm":
        state["x"] = _activation_rows(gen, rows, hidden).to(act)
        state["weight"] = (1 + 0.2 * _normal(gen, hidden)).to(_DTYPES[case["params"]])
        state["residual"] = _activation_rows(gen, rows, hidden).to(act) if case["residual"] else None
    elif op == "norm_grad":
        x = _activation_rows(gen, rows, hidden).to(act)
        state["weight"] = (1 + 0.2 * _normal(gen, hidden)).to(_DTYPES[case["params"]])
        state["dy"] = _gradient(gen, rows, hidden).to(act)
        state["dsummed"] = _gradient(gen, rows, hidden).to(act) if case["residual"] else None
        state["rstd"] = torch.rsqrt(x.float().square().mean(1) + _EPS)
        if case["records"]:
            state["packed"] = _records(x.float() * state["rstd"][:, None], case["block"], case["code"])
        else:
            state["x"] = x
    else:
        inner = case["inner"]
        state["weight"] = (_normal(gen, 2 * inner, hidden) * hidden ** -0.5).to(act)
        if op == "gated":
            x = _activation_rows(gen, rows, hidden)
            state["x"] = (x * torch.rsqrt(x.square().mean(1, keepdim=True) + _EPS)).to(act)
            state["bias"] = (0.2 * _normal(gen, 2 * inner)).to(act) if case["bias"] else None
        else:
            z = _normal(gen, rows, 2 * inner)
            z *= torch.exp(_normal(gen, 1, 2 * inner) * 0.3)
            state["packed"] = _records(z, case["block"], case["code"])
            state["dy"] = _gradient(gen, rows, inner).to(act)
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


def _kept(u, block, code):
    """What the records of u stand for, in bf16 (which holds it exactly)."""
    q, s = _quantise(u, block, code)
    return (q.float() * s).to(torch.bfloat16).view(u.shape)


def _values(packed, rows, hidden, block, code):
    """What a packed buffer stands for, as f32 [rows, hidden]."""
    records = packed.view(-1, block + 8)
    q = records[:, :block].contiguous().view(_FORMATS[code][2]).float()
    s = records[:, block + 4:].contiguous().view(torch.float32)
    return (q * s).view(rows, hidden)


_TANH_A, _TANH_B = math.sqrt(2 / math.pi), 0.044715


def _gate(g, activation):
    """act(g) and its slope."""
    if activation == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    if activation == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    t = torch.tanh(_TANH_A * (g + _TANH_B * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * _TANH_A * (1 + 3 * _TANH_B * g * g)


def _plain(state):
    case = state["case"]
    op, rows, block, code, act = case["op"], case["rows"], case["block"], case["code"], _DTYPES[case["dtype"]]
    if op == "norm":
        h = state["x"].float()
        if case["residual"]:
            h = (h + state["residual"].float()).to(act).float()
        rstd = torch.rsqrt(h.square().mean(1) + _EPS)
        xhat = h * rstd[:, None]
        y = xhat * state["weight"].float()
        out = {"y": _kept(y, block, code) if case["packed_y"] else y.to(act), "rstd": rstd}
        if case["residual"]:
            out["summed"] = h.to(act)
        if case["checkpoint"]:
            out["values"] = _kept(xhat, block, code)
        return out
    if op == "norm_grad":
        rstd = state["rstd"][:, None]
        xhat = _values(state["packed"], rows, case["hidden"], block, code) if case["records"] else state["x"].float() * rstd
        dy = state["dy"].float()
        a = dy * state["weight"].float()
        dx = rstd * (a - xhat * (a * xhat).mean(1, keepdim=True))
        if case["residual"]:
            dx = dx + state["dsummed"].float()
        return {"dx": dx.to(act), "dweight": (dy * xhat).sum(0).to(_DTYPES[case["params"]])}
    inner = case["inner"]
    if op == "gated":
        z = state["x"].float() @ state["weight"].float().t()
        if case["bias"]:
            z = z + state["bias"].float()
        out = {"y": (_gate(z[:, :inner], case["activation"])[0] * z[:, inner:]).to(act)}
        if case["checkpoint"]:
            out["values"] = _kept(z, block, code)
        return out
    z = _values(state["packed"], rows, 2 * inner, block, code)
    value, slope = _gate(z[:, :inner], case["activation"])
    dy, up = state["dy"].float(), z[:, inner:]
    dz = torch.cat([dy * up * slope, dy * value], 1)
    out = {"dz": dz.to(act), "dx": (dz @ state["weight"].float()).to(act)}
    if case["bias"]:
        out["dbias"] = dz.sum(0)
    if case["again"]:
        out["y"] = (value * up).to(act)
    return out


# ---------------------------------------------------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------------------------------------------------

def _framework(state):
    import fp8_compression_tensor_gb300 as taco

    case = state["case"]
    op, rows, hidden, block, code = case["op"], case["rows"], case["hidden"], case["block"], case["code"]
    if op == "norm":
        r = taco.rmsnorm(state["x"], state["weight"], eps=_EPS, residual=state["residual"], checkpoint=case["checkpoint"],
                         packed_y=case["packed_y"], block=block, code=code)
        out = {"y": taco.decompress(r.y, rows, hidden, block=block, variant="ds_only", code=code) if case["packed_y"] else r.y,
               "rstd": r.rstd}
        if case["residual"]:
            out["summed"] = r.summed
        if case["checkpoint"]:
            out["values"] = taco.decompress(r.packed, rows, hidden, block=block, variant="ds_only", code=code)
        return out
    if op == "norm_grad":
        g = taco.rmsnorm_backward(state["dy"], state["rstd"], state["weight"], x=state.get("x"), packed=state.get("packed"),
                                  dsummed=state["dsummed"], block=block, code=code)
        return {"dx": g.dx, "dweight": g.dweight}
    if op == "gated":
        r = taco.gated_linear(state["x"], state["weight"], state["bias"], activation=case["activation"],
                              checkpoint=case["checkpoint"], block=block, code=code)
        out = {"y": r.y}
        if case["checkpoint"]:
            out["values"] = taco.decompress(r.packed, rows, 2 * case["inner"], block=block, variant="ds_only", code=code)
        return out
    g = taco.gated_linear_backward(state["dy"], state["packed"], state["weight"], activation=case["activation"],
                                   bias_dtype=torch.float32 if case["bias"] else None, recompute=case["again"],
                                   block=block, code=code)
    out = {"dz": g.dz, "dx": g.dx}
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
    e = _BYTES[case["dtype"]]
    per_value = (block + 8) / block
    n = rows * hidden
    if op in ("norm", "norm_grad"):
        p = _BYTES[case["params"]] * hidden
        extra = n * e if case["residual"] else 0
        if op == "norm_grad":
            return {"bytes": 2 * n * e + (n * per_value if case["records"] else n * e) + extra + 4 * rows + 2 * p, "flops": 9 * n}
        # records are written, read again and returned as bf16 values
        eight = n * (2 * per_value + 2)
        return {"bytes": n * e + 2 * extra + 4 * rows + p + (eight if case["packed_y"] else n * e)
                + (eight if case["checkpoint"] else 0), "flops": 5 * n}
    m, weights = rows * case["inner"], 2 * case["inner"] * hidden
    bias = 2 * case["inner"] if case["bias"] else 0
    if op == "gated":
        kept = 2 * m * (2 * per_value + 2) if case["checkpoint"] else 0
        return {"bytes": e * (n + weights + m + bias) + kept, "flops": 2 * rows * weights}
    return {"bytes": e * (m + weights + 2 * m + n + (m if case["again"] else 0)) + 2 * m * per_value + 4 * bias,
            "flops": 2 * rows * weights}


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
    table, q = _code_table(code), torch.empty(bytes_.shape[0], block, dtype=torch.float64, device="cuda")
    for part in range(0, bytes_.shape[0], 1 << 18):   # (an index is eight bytes a value)
        q[part:part + (1 << 18)] = table[bytes_[part:part + (1 << 18), :block].long()]
    return q.mul_(scale).reshape(rows, hidden)


def _exact_gate(g, activation):
    """act(g) and its slope."""
    if activation == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if activation == "gelu":
        s = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * s, s + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(2 * inner)
    return g * s, s + g * 2 * s * torch.sigmoid(-2 * inner) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)


def exact(case, seed):
    state = prepare(case, seed)
    op, rows, hidden, block, code = case["op"], case["rows"], case["hidden"], case["block"], case["code"]
    if op == "norm":
        h, out = state["x"].double(), {}
        if case["residual"]:
            h = (h + state["residual"].double()).to(_DTYPES[case["dtype"]])
            out["summed"] = h
            h = h.double()
        rstd = 1 / torch.sqrt(torch.einsum("rc,rc->r", h, h) / hidden + _EPS)
        # a value next to a rounding tie takes either code by its 32-bit statistics
        out.update(y=None if case["packed_y"] else h * rstd[:, None] * state["weight"].double(), rstd=rstd)
        if case["checkpoint"]:
            out["values"] = None
        return out
    if op == "norm_grad":
        if case["records"]:
            xhat = _exact_values(state["packed"], rows, hidden, block, code)
        else:
            xhat = state["x"].double() * state["rstd"].double()[:, None]
        dy = state["dy"].double()
        a = dy * state["weight"].double()
        dx = (a - xhat * (torch.einsum("rc,rc->r", a, xhat) / hidden)[:, None]) * state["rstd"].double()[:, None]
        if case["residual"]:
            dx = dx + state["dsummed"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xhat)}
    inner = case["inner"]
    if op == "gated":
        weight, x = state["weight"].double(), state["x"].double()
        gate, up = torch.einsum("rh,ih->ri", x, weight[:inner]), torch.einsum("rh,ih->ri", x, weight[inner:])
        if case["bias"]:
            gate, up = gate + state["bias"][:inner].double(), up + state["bias"][inner:].double()
        out = {"y": _exact_gate(gate, case["activation"])[0] * up}
        if case["checkpoint"]:
            out["values"] = None   # as above, by the 32-bit sums
        return out
    z = _exact_values(state["packed"], rows, 2 * inner, block, code)
    value, slope = _exact_gate(z[:, :inner], case["activation"])
    dy, up, weight = state["dy"].double(), z[:, inner:], state["weight"].double()
    dgate, dup = dy * up * slope, dy * value
    out = {"dz": torch.cat([dgate, dup], 1),
           "dx": torch.einsum("ri,ih->rh", dgate, weight[:inner]) + torch.einsum("ri,ih->rh", dup, weight[inner:])}
    if case["bias"]:
        out["dbias"] = torch.cat([dgate.sum(0), dup.sum(0)])
    if case["again"]:
        out["y"] = value * up
    return out
