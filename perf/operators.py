"""What the 4-bit and normalisation operators are measured on.

Four operators of a layer that runs in 4 bits: the rounding of a tensor to microscaled 4-bit floating point
and back ("quantize"), the product of two such tensors ("product"), group norm with an activation over
channels-last tensors with its gradient ("norm", "norm_grad"), and the norm that writes 4-bit codes directly,
followed by the product that reads them ("norm_product").

A microscaled tensor of `rows` rows and `k` columns holds blocks of 32 consecutive columns: 4-bit codes (sign,
two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one power of two per block, 2^(s - 127).
Codes are stored [K1, rows, 64] bytes (K1 = ceil(k / 128), the lower columns in the lower half of a byte),
scales [K1, rows, 4] bytes; columns past k hold zeros.

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

#: The magnitudes that the eight codes without a sign stand for.
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one pooled feature vector on its way into a 4-bit head: the smallest call, where latency counts
        {"name": "quantize_one_vector", "op": "quantize", "rows": 1, "k": 2048, "type": "f16"},
        # odd sizes: rows that do not fill a block of 32 columns, nor 16 bytes
        {"name": "quantize_ragged_f32", "op": "quantize", "rows": 6241, "k": 997, "type": "f32"},
        # the res3 activations (28 x 28 x 512) of a large batch
        {"name": "quantize_res3_b256", "op": "quantize", "rows": 256 * 784, "k": 512, "type": "bf16"},
        # one new token through a projection: every weight is read for one row of sums
        {"name": "product_one_token", "op": "product", "m": 1, "n": 8192, "k": 8192, "type": "bf16", "act": "none",
         "bias": False, "residual": False},
        # the network's classifier (2048 -> 1000) over a batch, logits in float32; 1000 fills no power of two
        {"name": "product_head_b2048", "op": "product", "m": 2048, "n": 1000, "k": 2048, "type": "f32", "act": "none",
         "bias": True, "residual": False},
        # res3 conv3 (1x1, 128 -> 512 with shortcut and ReLU) in 4 bits: a short sum, bound by its output
        {"name": "product_res3_b64", "op": "product", "m": 64 * 784, "n": 512, "k": 128, "type": "bf16", "act": "relu",
         "bias": True, "residual": True},
        # a long prompt or a training-sized batch through a wide layer: bound by the matrix units
        {"name": "product_8192", "op": "product", "m": 8192, "n": 8192, "k": 8192, "type": "bf16", "act": "none",
         "bias": True, "residual": False},
        # one image's last feature map: latency
        {"name": "norm_one_image", "op": "norm", "n": 1, "hw": 49, "c": 2048, "groups": 32, "type": "bf16",
         "act": "relu"},
        # the res2 block output (56 x 56 x 256) of a batch, bound by memory
        {"name": "norm_res2_b128", "op": "norm", "n": 128, "hw": 3136, "c": 256, "groups": 32, "type": "bf16",
         "act": "silu"},
        # an odd image with groups of five channels, in float32, gradient
        {"name": "norm_grad_odd_f32", "op": "norm_grad", "n": 3, "hw": 1517, "c": 60, "groups": 12, "type": "f32",
         "act": "silu"},
        # the gradient at res3's size
        {"name": "norm_grad_res3_b64", "op": "norm_grad", "n": 64, "hw": 784, "c": 512, "groups": 32, "type": "bf16",
         "act": "silu"},
        # norm, activation and rounding in one, then the pointwise layer 512 -> 128 that reads the codes
        {"name": "norm_product_res3_b128", "op": "norm_product", "n": 128, "hw": 784, "c": 512, "groups": 32,
         "out": 128, "type": "bf16", "act": "silu"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "norm", "norm_grad", "norm_product"))
    kind = rng.choice(("f32", "bf16", "bf16", "f16"))
    act = rng.choice(("none", "relu", "silu"))
    if op == "quantize":
        k = _log(rng, 20, 8192)
        return {"op": op, "rows": _log(rng, 1, min(200000, 100_000_000 // k)), "k": k, "type": kind}
    if op == "product":
        n, k = _log(rng, 32, 8192), _log(rng, 32, 8192)
        # single rows often: a serving step
        m = rng.choice((1, _log(rng, 1, 64), _log(rng, 1, 8192), _log(rng, 64, 8192)))
        return {"op": op, "m": m, "n": n, "k": k, "type": kind, "act": act, "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5}
    groups = rng.choice((1, 4, 8, 16, 32, 32))
    c = groups * _log(rng, max(1, 32 // groups), 2048 // groups)
    hw = _log(rng, 1, 20000)
    n = _log(rng, 1, max(1, min(256, 50_000_000 // (hw * c))))
    case = {"op": op, "n": n, "hw": hw, "c": c, "groups": groups, "type": kind, "act": act}
    if op == "norm_product":
        case["out"] = _log(rng, 32, 2048)
    return case


# ---------------------------------------------------------------------------------------------- plain forms

def _quantize(x):
    """Codes and scales of x [rows, k] (any float type): the block's power of two is that of its largest
    magnitude, less two; a magnitude goes to the nearest level, to the even code where two are as near, and
    never past 6; a block that holds a NaN or an infinity has the scale 255, a NaN, and zero codes."""
    x = x.float()
    rows, k = x.shape
    k1 = (k + 127) // 128
    x = torch.nn.functional.pad(x, (0, 128 * k1 - k)).view(rows, k1, 4, 32)
    largest = x.abs().amax(-1)
    bad = ~torch.isfinite(largest)
    e = torch.frexp(torch.where(bad, 1.0, largest))[1]
    s = torch.where(largest > 0, (e + 124).clamp(0, 254), 0)
    s = torch.where(bad, 255, s)
    at = torch.where(bad[..., None], 0.0, torch.ldexp(x, 127 - s[..., None].clamp(max=254)))
    a = at.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int() + 8 * torch.signbit(at).int())
    code = code.view(rows, k1, 64, 2)
    codes = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
    return codes.permute(1, 0, 2).contiguous(), s.to(torch.uint8).permute(1, 0, 2).contiguous()


def _values(codes, scales, k):
    """float32 [rows, k] of codes [K1, rows, 64] and scales [K1, rows, 4]."""
    k1, rows, _ = codes.shape
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    c = codes.permute(1, 0, 2).int()
    v = level[torch.stack((c & 15, c >> 4), -1)].view(rows, k1, 4, 32)
    s = scales.permute(1, 0, 2).int()
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


def _norm(x, groups, weight, bias, act):
    """The activation of the group norm of x [n, hw, c] in float32, the means and the inverse deviations."""
    n, hw, c = x.shape
    g = x.float().view(n, hw, groups, c // groups)
    mean = g.mean((1, 3))
    g = g - mean[:, None, :, None]
    rstd = 1 / torch.sqrt((g * g).mean((1, 3)) + EPS)
    z = (g * rstd[:, None, :, None]).view(n, hw, c) * weight + bias
    return _act(z, act), mean, rstd


def _norm_grad(dy, x, mean, rstd, groups, weight, bias, act):
    n, hw, c = x.shape
    xhat = (x.float().view(n, hw, groups, -1) - mean[:, None, :, None]) * rstd[:, None, :, None]
    xhat = xhat.view(n, hw, c)
    dz = dy.float() * _act_grad(xhat * weight + bias, act)
    dweight, dbias = (dz * xhat).sum((0, 1)), dz.sum((0, 1))
    d = (dz * weight).view(n, hw, groups, -1)
    h = xhat.view(n, hw, groups, -1)
    dx = rstd[:, None, :, None] * (d - d.mean((1, 3), keepdim=True) - h * (d * h).mean((1, 3), keepdim=True))
    return dx.view(n, hw, c), dweight, dbias


# ---------------------------------------------------------------------------------------------- the cases

def _sixteen(kind):
    """What a layer that reads 4-bit codes hands on: 16 bits, of the features' type where that has 16."""
    return torch.float16 if kind == "f16" else torch.bfloat16


def _features(shape, gen):
    """A convolution's outputs before their norm: channels with their own mean and spread."""
    c = shape[-1]
    mean = torch.randn(c, generator=gen, device="cuda")
    spread = torch.exp(0.5 * torch.randn(c, generator=gen, device="cuda"))
    return torch.randn(shape, generator=gen, device="cuda") * spread + mean


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    st = dict(case)
    kind = TYPES[case["type"]]
    if case["op"] == "quantize":
        st["x"] = _features((case["rows"], case["k"]), gen).to(kind)
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        # activations after a ReLU-like gate, weights of a trained layer's scale
        st["a"] = _quantize(torch.nn.functional.silu(normal(m, k)))
        st["w"] = _quantize(normal(n, k) / math.sqrt(k))
        st["bias"] = normal(n) if case["bias"] else None
        st["residual"] = normal(m, n).to(kind) if case["residual"] else None
    else:
        n, hw, c, groups = case["n"], case["hw"], case["c"], case["groups"]
        st["x"] = _features((n, hw, c), gen).to(kind)
        st["weight"] = 1 + 0.2 * normal(c)
        st["bias"] = 0.3 * normal(c)
        if case["op"] == "norm_grad":
            _, st["mean"], st["rstd"] = _norm(st["x"], groups, st["weight"], st["bias"], "none")
            st["dy"] = normal(n, hw, c).to(kind)
        if case["op"] == "norm_product":
            st["w"] = _quantize(normal(case["out"], c) / math.sqrt(c))
            st["out_bias"] = normal(case["out"])
    return st


def _run_own(st):
    import convolution_int8_implicit_amd as ifx

    op = st["op"]
    if op == "quantize":
        return ifx.mx4_dequantize(ifx.mx4_quantize(st["x"]), torch.bfloat16)
    kind = TYPES[st["type"]]
    act = {"none": ifx.ACT_NONE, "relu": ifx.ACT_RELU, "silu": ifx.ACT_SILU}[st["act"]]
    if op == "product":
        a, w = ifx.Mx4(*st["a"], st["k"]), ifx.Mx4(*st["w"], st["k"])
        return ifx.mx4_matmul(a, w, st["bias"], st["residual"], act, kind)
    if op == "norm":
        return ifx.group_norm(st["x"], st["groups"], st["weight"], st["bias"], EPS, act)
    if op == "norm_grad":
        return ifx.group_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["groups"], st["weight"],
                                       st["bias"], act)
    q = ifx.group_norm_mx4(st["x"], st["groups"], st["weight"], st["bias"], EPS, act)
    return ifx.mx4_matmul(q, ifx.Mx4(*st["w"], st["c"]), st["out_bias"], None, ifx.ACT_NONE, _sixteen(st["type"]))


def run(state):
    if own:
        return _run_own(state)
    st, kind = state, TYPES[state["type"]]
    if st["op"] == "quantize":
        return _values(*_quantize(st["x"]), st["k"]).to(torch.bfloat16)
    if st["op"] == "product":
        y = _values(*st["a"], st["k"]) @ _values(*st["w"], st["k"]).t()
        if st["bias"] is not None:
            y = y + st["bias"]
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return _act(y, st["act"]).to(kind)
    if st["op"] == "norm":
        y, mean, rstd = _norm(st["x"], st["groups"], st["weight"], st["bias"], st["act"])
        return y.to(kind), mean, rstd
    if st["op"] == "norm_grad":
        dx, dweight, dbias = _norm_grad(st["dy"], st["x"], st["mean"], st["rstd"], st["groups"], st["weight"],
                                        st["bias"], st["act"])
        return dx.to(kind), dweight, dbias
    y = _norm(st["x"], st["groups"], st["weight"], st["bias"], st["act"])[0]
    codes, scales = _quantize(y.view(-1, st["c"]))
    y = _values(codes, scales, st["c"]) @ _values(*st["w"], st["c"]).t()
    return (y + st["out_bias"]).to(_sixteen(st["type"]))


def _code_bytes(rows, k):
    return rows * (-(-k // 32)) * 17


def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "quantize":
        rows, k = case["rows"], case["k"]
        return {"bytes": rows * k * (size + 2), "flops": 4 * rows * k}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        out = m * n * size * (2 if case["residual"] else 1)
        return {"bytes": _code_bytes(m, k) + _code_bytes(n, k) + out, "flops": 2 * m * n * k}
    values = case["n"] * case["hw"] * case["c"]
    if case["op"] == "norm":
        return {"bytes": 2 * values * size, "flops": 10 * values}
    if case["op"] == "norm_grad":
        return {"bytes": 3 * values * size, "flops": 25 * values}
    rows, c, out = case["n"] * case["hw"], case["c"], case["out"]
    return {"bytes": values * size + _code_bytes(out, c) + rows * out * 2, "flops": 14 * values + 2 * rows * c * out}


# ---------------------------------------------------------------------------------------------- 64 bits

def _exact_round(x):
    """The values that a float64 tensor [rows, k] has after the rounding to 4 bits, from the definition: of the
    levels of its block's power of two the nearest one, the one with the even code where two are as near."""
    rows, k = x.shape
    blocks = -(-k // 32)
    b = torch.zeros(rows, blocks * 32, dtype=torch.float64, device=x.device)
    b[:, :k] = x
    b = b.view(rows, blocks, 32)
    top = b.abs().max(-1, keepdim=True).values
    power = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    power = power - (torch.exp2(power) > top).double() * (top > 0) + (torch.exp2(power + 1) <= top).double()
    unit = torch.exp2(torch.where(top > 0, power - 2, -127.0).clamp(-127, 127))
    r = b.abs() / unit
    # spacing of the levels around r: 1/2 below 2, 1 up to 4, 2 above
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0)).double()
    v = (torch.round(r / step) * step).clamp(max=6.0)  # torch.round: halves to even, as the codes' last bit is
    return (torch.sign(b) * v * unit).view(rows, -1)[:, :k]


def _exact_values(q, k):
    codes, scales = (t.to(torch.int64) for t in q)
    k1, rows, _ = codes.shape
    low, high = codes % 16, codes // 16
    c = torch.stack((low, high), -1).reshape(k1, rows, 128)
    exponent, mantissa = (c // 2) % 4, c % 2
    magnitude = torch.where(exponent == 0, 0.5 * mantissa, torch.exp2(exponent.double() - 1) * (1 + 0.5 * mantissa))
    unit = torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    v = torch.where(c >= 8, -magnitude, magnitude) * unit
    return v.permute(1, 0, 2).reshape(rows, -1)[:, :k].contiguous()


def _exact_act(z, act):
    return {"none": lambda: z, "relu": lambda: torch.maximum(z, torch.zeros_like(z)),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def _exact_stats(x, groups):
    n, hw, c = x.shape
    g = x.transpose(1, 2).reshape(n, groups, -1)
    return g.mean(-1), 1 / torch.sqrt(g.var(-1, unbiased=False) + EPS)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_round(st["x"].double())
    if op == "product":
        y = torch.matmul(_exact_values(st["a"], case["k"]), _exact_values(st["w"], case["k"]).t())
        y = y if st["bias"] is None else y + st["bias"].double()
        y = y if st["residual"] is None else y + st["residual"].double()
        return _exact_act(y, case["act"])
    x, w, b = st["x"].double(), st["weight"].double(), st["bias"].double()
    groups, per = case["groups"], case["c"] // case["groups"]
    if op == "norm_grad":
        mean, rstd = (st[name].double().repeat_interleave(per, 1)[:, None] for name in ("mean", "rstd"))
        h = (x - mean) * rstd
        z = h * w + b
        s = torch.sigmoid(z)
        dz = st["dy"].double() * {"none": torch.ones_like(z), "relu": (z > 0).double(),
                                  "silu": s + z * s * (1 - s)}[case["act"]]
        d = dz * w

        def mean_of(t):
            return t.view(*t.shape[:2], groups, per).mean((1, 3)).repeat_interleave(per, 1)[:, None]

        return rstd * (d - mean_of(d) - h * mean_of(d * h)), (dz * h).sum((0, 1)), dz.sum((0, 1))
    mean, rstd = _exact_stats(x, groups)
    z = (x - mean.repeat_interleave(per, 1)[:, None]) * rstd.repeat_interleave(per, 1)[:, None] * w + b
    y = _exact_act(z, case["act"])
    if op == "norm":
        return y, mean, rstd
    q = _exact_round(y.view(-1, case["c"]))
    return q @ _exact_values(st["w"], case["c"]).t() + st["out_bias"].double()
