"""What the 8-bit feed-forward operators are measured on.

The operators of a feed-forward layer in 8-bit floating point, for serving and for training: the product of two
8-bit tensors ("product", also from wider tensors that are rounded on the way, as a weight's gradient is), root mean
square norm with the residual's addition and its gradient ("norm", "norm_grad"), the gated pair of projections
act(x G^T) (x U^T) behind a norm that writes 8 bits ("norm_gated"), its gradient ("gated_grad"), and the pair that
writes 8 bits with the product and the residual behind it ("feed").

An 8-bit tensor of `rows` rows and k columns holds blocks of 128 consecutive columns: one byte a column, sign, exponent
and mantissa of 4 and 3 bits ("e4m3", up to 448, no infinity) or of 5 and 2 ("e5m2", up to 57344), and one power of
two per block, 2^(s - 127).  Codes are stored [K1, rows, 128] bytes (K1 = ceil(k / 128)), scales
[ceil(K1 / 4), rows, 4] bytes; columns past k hold zeros.

`run` computes each operator in elementary torch operations in 32 bits, or, where `own` is true, by the calls
that a program makes of convolution_int8_implicit_amd.
"""
import math

import torch

own = False

#: float32 and the 16-bit types by the name that a case gives them.
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5

#: The 8-bit types: torch's, the exponent of their largest power of two, mantissa bits, their smallest exponent.
FORMATS = {"e4m3": (torch.float8_e4m3fn, 8, 3, -6), "e5m2": (torch.float8_e5m2, 15, 2, -14)}


def listed():
    return [
        # one new token through a projection: every weight is read for one row of sums
        {"name": "product_one_token", "op": "product", "m": 1, "n": 8192, "k": 8192, "type": "bf16", "side": "codes",
         "format": "e4m3", "act": "none", "bias": False, "residual": False},
        # a weight's gradient dy^T x of an odd layer over an odd number of tokens, to float32: both tensors are
        # transposed and rounded in the call, dy to five exponent bits
        {"name": "product_weight_grad", "op": "product", "m": 1000, "n": 2048, "k": 6241, "type": "f32",
         "side": "columns", "format": "e5m2", "act": "none", "bias": False, "residual": False},
        # a long prompt or a training-sized batch through a wide layer: bound by the matrix units
        {"name": "product_8192", "op": "product", "m": 8192, "n": 8192, "k": 8192, "type": "bf16", "side": "codes",
         "format": "e4m3", "act": "none", "bias": True, "residual": False},
        # odd rows in float32 that fill neither a block of 128 nor 16 bytes
        {"name": "norm_odd_f32", "op": "norm", "rows": 6241, "c": 997, "type": "f32", "residual": False},
        # the tokens of a long prompt in a wide layer, with the residual: bound by memory
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "c": 8192, "type": "bf16", "residual": True},
        # a small batch's gradient, rows shorter than a workgroup
        {"name": "norm_grad_odd_f16", "op": "norm_grad", "rows": 1517, "c": 510, "type": "f16", "past": False},
        # a training batch's gradient with the gradient that comes past the norm
        {"name": "norm_grad_batch", "op": "norm_grad", "rows": 16384, "c": 4096, "type": "bf16", "past": True},
        # sizes that fill no tile: the norm that rounds to 8 bits, then the gated projections
        {"name": "norm_gated_odd", "op": "norm_gated", "m": 333, "n": 1000, "k": 997, "type": "f16", "act": "silu"},
        # a training batch's gradient at the gate and the value, of odd sizes and of whole tiles
        {"name": "gated_grad_odd", "op": "gated_grad", "m": 1517, "n": 2500, "k": 510, "type": "f32", "act": "silu"},
        {"name": "gated_grad_batch", "op": "gated_grad", "m": 4096, "n": 8192, "k": 2048, "type": "bf16", "act": "silu"},
        # a serving step of one token through both projections and back: latency and the weights' bytes
        {"name": "feed_one_token", "op": "feed", "m": 1, "n": 8192, "k": 2048, "type": "bf16", "act": "silu"},
        # a prompt through them
        {"name": "feed_prompt", "op": "feed", "m": 4096, "n": 8192, "k": 2048, "type": "bf16", "act": "silu"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("product", "product", "norm", "norm_grad", "norm_gated", "gated_grad", "feed"))
    kind = rng.choice(("f32", "bf16", "bf16", "f16"))
    act = rng.choice(("none", "relu", "silu", "silu"))
    # single rows often: a serving step
    m = rng.choice((1, _log(rng, 1, 64), _log(rng, 1, 4096), _log(rng, 64, 4096)))
    if op == "product":
        side = rng.choice(("codes", "codes", "columns"))
        fmt = rng.choice(("e4m3", "e5m2"))
        if side == "columns":
            return {"op": op, "m": _log(rng, 32, 4096), "n": _log(rng, 32, 4096), "k": _log(rng, 1, 16384), "type": kind,
                    "side": side, "format": fmt, "act": "none", "bias": False, "residual": rng.random() < 0.5}
        return {"op": op, "m": m * rng.choice((1, 2)), "n": _log(rng, 32, 8192), "k": _log(rng, 32, 8192), "type": kind,
                "side": side, "format": fmt, "act": act, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    if op in ("norm", "norm_grad"):
        c = _log(rng, 16, 16384)
        case = {"op": op, "rows": _log(rng, 1, min(65536, 60_000_000 // c)), "c": c, "type": kind}
        case["residual" if op == "norm" else "past"] = rng.random() < 0.5
        return case
    if op == "gated_grad" and act == "relu":
        act = "silu"  # a ReLU's slope is decided by the last bit where its argument is next to zero
    if op != "gated_grad" and kind == "f32":
        kind = "bf16"  # what is behind a rounding to 8 bits is handed on in 16
    return {"op": op, "m": m, "n": _log(rng, 32, 8192), "k": _log(rng, 32, 4096), "type": kind, "act": act}


# ---------------------------------------------------------------------------------------------- plain forms

def _quantize(x, fmt="e4m3"):
    """Codes and scales of x [rows, k] (any float type): the block's power of two is the smallest one under which its
    largest magnitude, in units of it, is at most the type's largest value, and at least 2^-127; codes are rounded to
    nearest, halves to even; a block that holds a NaN or an infinity has the scale 255, a NaN, and zero codes."""
    dtype, top_exponent, _, _ = FORMATS[fmt]
    x = x.float()
    rows, k = x.shape
    k1 = (k + 127) // 128
    x = torch.nn.functional.pad(x, (0, 128 * k1 - k)).view(rows, k1, 128)
    largest = x.abs().amax(-1)
    bad = ~torch.isfinite(largest)
    f, e = torch.frexp(torch.where(bad, 1.0, largest))
    s = torch.where(largest > 0, (e - 1 - top_exponent + 127 + (f > 0.875).int()).clamp(0, 254), 0)
    s = torch.where(bad, 255, s)
    at = torch.where(bad[..., None], 0.0, torch.ldexp(x, 127 - s[..., None].clamp(max=254)))
    codes = at.to(dtype).view(torch.uint8).permute(1, 0, 2).contiguous()
    k4 = (k1 + 3) // 4
    s = torch.nn.functional.pad(s, (0, 4 * k4 - k1)).to(torch.uint8)
    return codes, s.view(rows, k4, 4).permute(1, 0, 2).contiguous()


def _values(codes, scales, k, fmt="e4m3"):
    """float32 [rows, k] of codes [K1, rows, 128] and scales [ceil(K1 / 4), rows, 4]."""
    k1, rows, _ = codes.shape
    v = codes.view(FORMATS[fmt][0]).float().permute(1, 0, 2)
    s = scales.permute(1, 0, 2).reshape(rows, -1)[:, :k1].int()
    v = torch.ldexp(v, (s - 127)[..., None])
    v = torch.where((s == 255)[..., None], math.nan, v)
    return v.reshape(rows, 128 * k1)[:, :k]


def _act(z, act):
    return z.clamp(min=0) if act == "relu" else z * (1 / (1 + torch.exp(-z))) if act == "silu" else z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _norm(x, residual, weight):
    """The norm of x + residual [rows, c] in float32, the sum in x's type and the inverse root mean squares."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    f = h.float()
    rstd = 1 / torch.sqrt((f * f).mean(-1) + EPS)
    return f * rstd[:, None] * weight, h, rstd


def _norm_grad(dy, h, rstd, weight, past):
    xhat = h.float() * rstd[:, None]
    d = dy.float()
    dweight = (d * xhat).sum(0)
    d = d * weight
    dx = rstd[:, None] * (d - xhat * (d * xhat).mean(-1, keepdim=True))
    return dx if past is None else dx + past.float(), dweight


# ---------------------------------------------------------------------------------------------- the cases

def _features(rows, c, gen):
    """A residual stream: channels of their own spread, some of them far wider than the rest."""
    spread = torch.exp(0.7 * torch.randn(c, generator=gen, device="cuda"))
    return torch.randn((rows, c), generator=gen, device="cuda") * spread


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def weights(n, k):
        """A trained layer's weights, rounded once."""
        return _quantize(normal(n, k) / math.sqrt(k))

    st, kind, op = dict(case), TYPES[case["type"]], case["op"]
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        if case["side"] == "columns":
            # gradients of a mean over the tokens, and activations
            st["a"] = (normal(k, m) / k).to(kind)
            st["w"] = torch.nn.functional.silu(normal(k, n)).to(kind)
        else:
            st["a"] = _quantize(torch.nn.functional.silu(normal(m, k)), case["format"])
            st["w"] = weights(n, k)
        st["b"] = normal(n) if case["bias"] else None
        st["r"] = normal(m, n).to(kind) if case["residual"] else None
    elif op in ("norm", "norm_grad"):
        rows, c = case["rows"], case["c"]
        st["x"] = _features(rows, c, gen).to(kind)
        st["weight"] = 1 + 0.2 * normal(c)
        if op == "norm":
            st["r"] = _features(rows, c, gen).to(kind) if case["residual"] else None
        else:
            st["rstd"] = _norm(st["x"], None, st["weight"])[2]
            st["dy"] = normal(rows, c).to(kind)
            st["dh"] = normal(rows, c).to(kind) if case["past"] else None
    else:
        m, n, k = case["m"], case["n"], case["k"]
        st["gate"], st["up"] = weights(n, k), weights(n, k)
        if op == "norm_gated":
            st["x"], st["r"] = _features(m, k, gen).to(kind), _features(m, k, gen).to(kind)
            st["weight"] = 1 + 0.2 * normal(k)
        else:
            st["x"] = _quantize(normal(m, k))
        if op == "gated_grad":
            st["dy"] = normal(m, n).to(kind)
        if op == "feed":
            st["down"], st["r"] = weights(k, n), normal(m, k).to(kind)
    return st


def _run_own(st):
    import convolution_int8_implicit_amd as ifx

    op, kind = st["op"], TYPES[st["type"]]
    formats = {"e4m3": ifx.FP8_E4M3, "e5m2": ifx.FP8_E5M2}
    acts = {"none": ifx.ACT_NONE, "relu": ifx.ACT_RELU, "silu": ifx.ACT_SILU}
    if op == "product":
        fmt = formats[st["format"]]
        if st["side"] == "columns":
            a, w = ifx.fp8_quantize_t(st["a"], fmt), ifx.fp8_quantize_t(st["w"])
        else:
            a, w = ifx.Fp8(*st["a"], st["k"], fmt), ifx.Fp8(*st["w"], st["k"], ifx.FP8_E4M3)
        return ifx.fp8_matmul(a, w, st["b"], st["r"], acts[st["act"]], kind)
    if op == "norm":
        return ifx.rms_norm(st["x"], st["weight"], st["r"], EPS)
    if op == "norm_grad":
        return ifx.rms_norm_backward(st["dy"], st["x"], st["rstd"], st["weight"], st["dh"])
    act, e4m3, k = acts[st["act"]], ifx.FP8_E4M3, st["k"]
    gate, up = ifx.Fp8(*st["gate"], k, e4m3), ifx.Fp8(*st["up"], k, e4m3)
    if op == "norm_gated":
        q, h, _ = ifx.rms_norm_fp8(st["x"], st["weight"], st["r"], EPS)
        return ifx.gated(q, gate, up, act, kind), h
    x = ifx.Fp8(*st["x"], k, e4m3)
    if op == "feed":
        q = ifx.gated_fp8(x, gate, up, act)
        return ifx.fp8_matmul(q, ifx.Fp8(*st["down"], st["n"], e4m3), None, st["r"], ifx.ACT_NONE, kind)
    return ifx.gated_backward(st["dy"], x, gate, up, act)


def run(state):
    if own:
        return _run_own(state)
    st, op, kind = state, state["op"], TYPES[state["type"]]
    if op == "product":
        k, fmt = st["k"], st["format"]
        if st["side"] == "columns":
            a, w = _quantize(st["a"].t(), fmt), _quantize(st["w"].t())
        else:
            a, w = st["a"], st["w"]
        y = _values(*a, k, fmt) @ _values(*w, k).t()
        if st["b"] is not None:
            y = y + st["b"]
        if st["r"] is not None:
            y = y + st["r"].float()
        return _act(y, st["act"]).to(kind)
    if op == "norm":
        y, h, rstd = _norm(st["x"], st["r"], st["weight"])
        return y.to(kind), h, rstd
    if op == "norm_grad":
        dx, dweight = _norm_grad(st["dy"], st["x"], st["rstd"], st["weight"], st["dh"])
        return dx.to(kind), dweight
    if op == "norm_gated":
        y, h, _ = _norm(st["x"], st["r"], st["weight"])
        x = _values(*_quantize(y), st["k"])
    else:
        x = _values(*st["x"], st["k"])
    g, u = x @ _values(*st["gate"], st["k"]).t(), x @ _values(*st["up"], st["k"]).t()
    if op == "gated_grad":
        dy = st["dy"].float()
        return (dy * u * _act_grad(g, st["act"])).to(kind), (dy * _act(g, st["act"])).to(kind)
    y = _act(g, st["act"]) * u
    if op == "norm_gated":
        return y.to(kind), h
    y = _values(*_quantize(y), st["n"]) @ _values(*st["down"], st["n"]).t()
    return (y + st["r"].float()).to(kind)


def _code_bytes(rows, k):
    return rows * (k + -(-k // 128))


def work(case):
    size, op = SIZE[case["type"]], case["op"]
    if op in ("norm", "norm_grad"):
        values = case["rows"] * case["c"]
        if op == "norm":
            return {"bytes": values * size * (4 if case["residual"] else 2), "flops": 5 * values}
        return {"bytes": values * size * (4 if case["past"] else 3), "flops": 10 * values}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "product":
        out = m * n * size * (2 if case["residual"] else 1)
        read = (m + n) * k * size if case["side"] == "columns" else _code_bytes(m, k) + _code_bytes(n, k)
        return {"bytes": read + out, "flops": 2 * m * n * k}
    weights = 2 * _code_bytes(n, k)
    if op == "gated_grad":
        return {"bytes": _code_bytes(m, k) + weights + 3 * m * n * size, "flops": 4 * m * n * k}
    if op == "norm_gated":
        return {"bytes": 3 * m * k * size + weights + m * n * size, "flops": 4 * m * n * k}
    return {"bytes": _code_bytes(m, k) + weights + _code_bytes(k, n) + 2 * m * k * size, "flops": 6 * m * n * k}


# ---------------------------------------------------------------------------------------------- 64 bits

def _floor_log2(v):
    power = torch.floor(torch.log2(v))
    power = power - (torch.exp2(power) > v).double()
    return power + (torch.exp2(power + 1) <= v).double()


def _exact_round(x, fmt="e4m3"):
    """The values that a float64 tensor [rows, k] has after the rounding to 8 bits, from the definition."""
    _, _, bits, lowest = FORMATS[fmt]
    most = {"e4m3": 448.0, "e5m2": 57344.0}[fmt]
    rows, k = x.shape
    blocks = -(-k // 128)
    b = torch.zeros(rows, blocks * 128, dtype=torch.float64, device=x.device)
    b[:, :k] = x
    b = b.view(rows, blocks, 128)
    top = b.abs().max(-1, keepdim=True).values
    # the smallest power of two with top <= most * 2^power
    power = _floor_log2(torch.where(top > 0, top / most, 1.0))
    power = power + (torch.exp2(power) * most < top).double()
    unit = torch.exp2(torch.where(top > 0, power, -127.0).clamp(min=-127.0))
    r = b.abs() / unit
    step = torch.exp2(_floor_log2(r.clamp(min=2.0 ** lowest)) - bits)
    v = torch.round(r / step) * step  # torch.round: halves to even, as the codes' last bit is
    return (torch.sign(b) * v * unit).view(rows, -1)[:, :k]


def _exact_values(q, k, fmt="e4m3"):
    _, _, bits, lowest = FORMATS[fmt]
    codes, scales = (t.to(torch.int64) for t in q)
    k1, rows, _ = codes.shape
    exponent, mantissa = (codes >> bits) & (2 ** (7 - bits) - 1), (codes & (2 ** bits - 1)).double() / 2 ** bits
    power = torch.exp2((exponent - 1 + lowest).double())
    v = torch.where(exponent == 0, mantissa * 2.0 ** lowest, (1 + mantissa) * power)
    v = torch.where(codes >= 128, -v, v).permute(1, 0, 2)
    unit = torch.exp2(scales.permute(1, 0, 2).reshape(rows, -1)[:, :k1].double() - 127)
    return (v * unit[..., None]).reshape(rows, -1)[:, :k].contiguous()


def _exact_act(z, act):
    return {"none": lambda: z, "relu": lambda: torch.maximum(z, torch.zeros_like(z)),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "product":
        k, fmt = case["k"], case["format"]
        if case["side"] == "columns":
            a, w = _exact_round(st["a"].double().t(), fmt), _exact_round(st["w"].double().t())
        else:
            a, w = _exact_values(st["a"], k, fmt), _exact_values(st["w"], k)
        y = torch.matmul(a, w.t())
        y = y if st["b"] is None else y + st["b"].double()
        y = y if st["r"] is None else y + st["r"].double()
        return _exact_act(y, case["act"])
    if op in ("norm", "norm_gated"):
        whole = st["x"].double() if st["r"] is None else st["x"].double() + st["r"].double()
        h = whole.to(st["x"].dtype).double()  # the norm is that of the sum as it is kept
        rstd = (h.square().sum(-1) / h.shape[-1] + EPS).rsqrt()
        y = h * rstd[:, None] * st["weight"].double()
        if op == "norm":
            return y, whole, rstd
    if op == "norm_grad":
        rstd = st["rstd"].double()[:, None]
        h, dy, w = st["x"].double(), st["dy"].double(), st["weight"].double()
        inner = (dy * w * h).sum(-1, keepdim=True) / h.shape[-1]
        dx = rstd * dy * w - rstd ** 3 * h * inner
        return dx if st["dh"] is None else dx + st["dh"].double(), (dy * h * rstd).sum(0)
    k = case["k"]
    x = _exact_round(y) if op == "norm_gated" else _exact_values(st["x"], k)
    g, u = torch.matmul(x, _exact_values(st["gate"], k).t()), torch.matmul(x, _exact_values(st["up"], k).t())
    if op == "norm_gated":
        return _exact_act(g, case["act"]) * u, whole
    if op == "feed":
        y = _exact_round(_exact_act(g, case["act"]) * u)
        return torch.matmul(y, _exact_values(st["down"], case["n"]).t()) + st["r"].double()
    s = torch.sigmoid(g)
    slope = {"none": torch.ones_like(g), "relu": (g > 0).double(), "silu": s + g * s * (1 - s)}[case["act"]]
    dy = st["dy"].double()
    return dy * u * slope, dy * _exact_act(g, case["act"])
