"""The gated pair of projections of 8-bit tensors, its 8-bit form and its gradient: refusals (CPU) and the kernels
against the 64-bit reference (GPU).

Bounds: with t the bound of a projection's sum (tests/test_fp8.py) times the sum of its terms' magnitudes, at the gate tg
and at the other tu, act(g) u is off by at most |act(g)| tu + 1.1 tg (|u| + tu), for SiLU also (|g| + 4) 2^-22 |act(g) u|
for its exponential and division, and 2^-23 of itself for the product; then one rounding to the type.  The gradient's two
results likewise, with |act'| <= 1.1 and |act''| <= 0.5.  On whole numbers every sum is exact.
"""
import ctypes

import numpy as np
import pytest
import torch

import convolution_int8_implicit_amd as ifx
from oracle import lowp
from test_fp8 import integer_codes, random_codes, same_codes, sum_bound, tensor_of
from test_fp8 import cuda64, whole_excess
from test_mx4 import TYPES, excess, f64, note

ACTS = {"none": 0, "relu": 1, "silu": 2}


# ------------------------------------------------------------------------------------------ CPU

def test_refusals_need_no_device():
    L = ifx.lib()
    fake, odd, half = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001), ctypes.c_void_p(0x100002)
    names = ("x", "xs", "g", "gs", "u", "us")

    def desc(m=200, n=3, k=4, t=1, act=2, ld_y=3, ld_up=3, ld_dy=3):
        return ctypes.byref(ifx.GatedDesc(m, n, k, t, act, ld_y, ld_up, ld_dy))

    def forward(y=fake, **kw):
        ptr = {s: kw.pop(s, fake) for s in names}
        return L.ifx_gated(desc(**kw), *ptr.values(), y, None)

    def eight(codes=fake, scales=fake, ws=fake, ws_bytes=1 << 30, **kw):
        ptr = {s: kw.pop(s, fake) for s in names}
        return L.ifx_gated_fp8(desc(**kw), *ptr.values(), codes, scales, ws, ws_bytes, None)

    def backward(dy=fake, dgate=fake, dup=fake, **kw):
        ptr = {s: kw.pop(s, fake) for s in names}
        return L.ifx_gated_backward(desc(**kw), dy, *ptr.values(), dgate, dup, None)
    assert L.ifx_gated(None, *[fake] * 7, None) == 1 and L.ifx_gated_fp8(None, *[fake] * 9, 0, None) == 1
    assert L.ifx_gated_backward(None, *[fake] * 10) == 1
    for call in (forward, eight, backward):
        for s in names:
            assert call(**{s: None}) == 1, s
            assert call(**{s: half}) == 4, s
        assert call(t=3) == 3 and call(act=3) == 3
        assert call(m=-1) == 2 and call(n=-1) == 2 and call(k=0) == 2
        assert call(m=1 << 18, n=1 << 18, ld_y=1 << 18, ld_up=1 << 18, ld_dy=1 << 18) == 2
        assert call(m=0, x=None) == 0 and call(n=0, ld_y=0, ld_up=0, ld_dy=0, g=None) == 0
    assert forward(y=None) == 1 and forward(y=odd) == 4 and forward(ld_y=2) == 2
    assert eight(codes=None) == 1 and eight(scales=None) == 1 and eight(codes=half) == 4
    assert eight(ld_y=0, codes=None) == 1  # its pitch is not looked at
    # up to 16 rows pass through the workspace
    assert L.ifx_gated_workspace_bytes(desc(m=16, n=1000)) == 16 * 1000 * 4
    assert L.ifx_gated_workspace_bytes(desc(m=17, n=1000)) == 0 and L.ifx_gated_workspace_bytes(desc(k=0)) == 0
    assert eight(m=4, ws_bytes=4 * 3 * 4 - 1) == 5 and eight(m=4, ws=None) == 1 and eight(m=4, ws=half) == 4
    for s in ("dy", "dgate", "dup"):
        assert backward(**{s: None}) == 1 and backward(**{s: odd}) == 4
    assert backward(ld_y=2) == 2 and backward(ld_up=2) == 2 and backward(ld_dy=2) == 2


def test_binding_refusals_need_no_device(monkeypatch):
    monkeypatch.setattr(ifx, "_on_device", lambda *ts: 0)
    monkeypatch.setattr(ifx, "_raw_stream", lambda stream, index: 0)

    def fp8(rows, k, fmt=0):
        return ifx.fp8_empty(rows, k, fmt, device="meta")

    def dy(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="meta")
    good = (fp8(4, 32), fp8(6, 32), fp8(6, 32))
    for bad in ((fp8(4, 33), *good[1:]), (good[0], fp8(5, 32), good[2]), (*good[:2], fp8(6, 31)), (fp8(4, 32, 1), *good[1:]),
                (good[0], fp8(6, 32, 1), good[2]), (*good[:2], fp8(6, 32, 1))):
        for call in (ifx.gated, ifx.gated_fp8, lambda *q: ifx.gated_backward(dy(4, 6), *q)):
            with pytest.raises(ValueError):
                call(*bad)
    with pytest.raises(ValueError):
        ifx.gated(*good, out=dy(4, 5))
    with pytest.raises(ValueError):
        ifx.gated_fp8(*good, out=fp8(4, 5))
    with pytest.raises(ValueError):
        ifx.gated_fp8(*good, out=fp8(4, 6, 1))
    with pytest.raises(ValueError):
        ifx.gated_backward(dy(6, 4), *good)
    with pytest.raises(ValueError):
        ifx.gated_backward(dy(4, 6), *good, out=(dy(4, 6), dy(4, 6, dtype=torch.float16)))
    with pytest.raises(TypeError):
        ifx.gated(*good, dtype=torch.int8)


def test_gradients_in_one_memory_are_refused(monkeypatch):
    monkeypatch.setattr(ifx, "_on_device", lambda *ts: 0)
    monkeypatch.setattr(ifx, "_raw_stream", lambda stream, index: 0)

    class Lib:
        def ifx_gated_backward(self, *args):
            return 0
    monkeypatch.setattr(ifx, "lib", Lib)
    q = [ifx.fp8_empty(rows, 32, device="meta") for rows in (4, 6, 6)]
    dy, other, wide = torch.zeros(4, 6), torch.zeros(4, 6), torch.zeros(4, 20)
    for out in ((dy, other), (other, dy), (wide[:, :6], wide[:, 6:12]), (wide[:, 14:], wide[:, :6])):
        assert ifx.gated_backward(dy, *q, out=out) is out
    for out in ((dy, dy), (other, other), (wide[:, :6], wide[:, 5:11]), (wide[:, 9:15], wide[:, 4:10])):
        with pytest.raises(ValueError, match="share"):
            ifx.gated_backward(dy, *q, out=out)


# ------------------------------------------------------------------------------------------ GPU

def gated_case(m, n, k, seed):
    rng = np.random.default_rng(seed)
    # sums of a few units: codes reach 2^8
    low = 122 - int(np.ceil(np.log2(k + 1) / 4))
    return tuple(random_codes(rng, rows, k, 0, low - 3, low + 1) for rows in (m, n, n)), rng


def bounds(q, k, act, kind):
    """(y, g, u, tolerance of y, tg, tu)."""
    y, g, u, sg, su = lowp.gated(*q, k, act)
    b = sum_bound(k, kind)
    tg, tu = b * sg, b * su
    a = np.abs(lowp.act(g, act))
    tol = a * tu + 1.1 * tg * (np.abs(u) + tu) + 2.0 ** -23 * np.abs(y)
    if act == 2:
        tol = tol + (np.abs(g) + 4) * 2.0 ** -22 * np.abs(y)
    return y, g, u, tol, tg, tu


def check_fp8(got, y, tol, k):
    """Codes of values within tol of y: the scale that such values' largest has, and under it codes between those of
    y - tol and y + tol."""
    codes, scales = got.codes.cpu().numpy(), got.scales.cpu().numpy()
    rows = y.shape[0]
    k1 = (k + 127) // 128
    s = scales.transpose(1, 0, 2).reshape(rows, -1)[:, :k1].astype(np.int64)
    assert not scales.transpose(1, 0, 2).reshape(rows, -1)[:, k1:].any()
    v = lowp.fp8_values(codes, scales, k1 * 128)
    assert not codes.transpose(1, 0, 2).reshape(rows, -1)[:, k:].any()

    def padded(t):
        out = np.zeros((rows, k1 * 128))
        out[:, :k] = t
        return out.reshape(rows, k1, 128)
    y, tol, v = padded(y), padded(tol), v.reshape(rows, k1, 128)
    top = np.abs(y).max(-1)
    t = tol.max(-1)
    for sign in (-1, 1):  # the scales of the largest and the smallest block
        edge = np.maximum(top + sign * t, 0)
        e = lowp.fp8_quantize(edge.reshape(-1, 1))[1][0, :, 0].reshape(rows, k1)
        assert (s <= e).all() if sign > 0 else (s >= e).all()
    unit = np.ldexp(1.0, s - 127)[..., None]

    def rounded(t):
        t = np.clip(t / unit, -448, 448)
        return np.sign(t) * lowp.FP8[0][lowp._fp8_nearest(np.abs(t), 0)] * unit
    assert (v >= rounded(y - tol)).all() and (v <= rounded(y + tol)).all()


SHAPES = [(1, 1, 1), (1, 40, 2048), (1, 33, 4224), (2, 17, 33), (3, 500, 4100), (5, 1000, 130), (7, 260, 2200), (16, 16, 128),
          (17, 31, 129), (33, 65, 640), (64, 128, 256), (65, 130, 96), (100, 300, 1000), (130, 257, 385), (257, 129, 512),
          (300, 520, 64), (1900, 850, 700), (2050, 1025, 300), (2111, 2130, 900), (4097, 2100, 130)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forms_and_gradient(m, n, k):
    for i, (kind, act) in enumerate((("f32", "silu"), ("bf16", "relu"), ("f16", "none"), ("bf16", "silu"))):
        if m * n > 2_000_000 and i in (1, 2):
            continue
        note(f"gated {m} x {n} x {k} {kind} {act}")
        q, rng = gated_case(m, n, k, m + 3 * n + 7 * k + i)
        X, G, U = (tensor_of(t, k) for t in q)
        y, g, u, tol, tg, tu = bounds(q, k, ACTS[act], kind)
        if kind == "f16":
            assert np.abs(y).max() < 30000
        got = ifx.gated(X, G, U, ACTS[act], TYPES[kind])
        assert got.shape == (m, n) and got.dtype == TYPES[kind]
        assert excess(f64(got), y, tol, kind) == 0
        if kind == "bf16":
            check_fp8(ifx.gated_fp8(X, G, U, ACTS[act]), y, tol, n)
        dy = torch.from_numpy(rng.standard_normal((m, n))).to(TYPES[kind])
        dgate, dup = ifx.gated_backward(dy.cuda(), X, G, U, ACTS[act])
        d = f64(dy)
        eg, eu = lowp.gated_backward(d, g, u, ACTS[act])
        more = (np.abs(g) + 4) * 2.0 ** -22 if act == "silu" else 0.0
        # |s (1 - s) g| < 0.23, so 1 + z (1 - s) of the slope loses at most (|g| + 4) 2^-22 of what it multiplies
        tol_g = np.abs(d) * (1.1 * tu + 0.5 * tg * (np.abs(u) + tu) + (1.1 * more + 2.0 ** -22) * (np.abs(u) + tu))
        if act == "relu":  # the corner is decided by the computed projection
            eg = np.where(np.abs(g) <= tg, 0.0, eg)
            tol_g = tol_g + np.where(np.abs(g) <= tg, np.abs(d) * (np.abs(u) + tu), 0.0)
        tol_u = np.abs(d) * (1.1 * tg + (more + 2.0 ** -22) * np.abs(lowp.act(g, ACTS[act])))
        assert excess(f64(dgate), eg, tol_g, kind) == 0
        assert excess(f64(dup), eu, tol_u, kind) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_whole_numbers(m, n, k):
    """Sums and products that every step leaves exact: values, codes and gradients bit for bit."""
    rng = np.random.default_rng(m * n + k)
    note(f"gated whole numbers {m} x {n} x {k}")
    most = 1 if k > 1000 else 2
    q = tuple(integer_codes(rng, rows, k, 0, most) for rows in (m, n, n))
    X, G, U = (tensor_of(t, k) for t in q)
    for act in (0, 1):
        y, g, u, _, _ = lowp.gated(*q, k, act)
        assert np.abs(y).max() < 2 ** 24
        for kind in ("bf16", "f32"):
            assert torch.equal(ifx.gated(X, G, U, act, TYPES[kind]).cpu(), torch.from_numpy(y).to(TYPES[kind]))
        assert same_codes(ifx.gated_fp8(X, G, U, act), lowp.fp8_quantize(y))
        d = rng.integers(-2, 3, (m, n)).astype(np.float64)
        for kind in ("f16", "f32"):
            dgate, dup = ifx.gated_backward(torch.from_numpy(d).to(TYPES[kind]).cuda(), X, G, U, act)
            eg, eu = lowp.gated_backward(d, g, u, act)
            assert torch.equal(dgate.cpu(), torch.from_numpy(eg + 0.0).to(TYPES[kind]))
            assert torch.equal(dup.cpu(), torch.from_numpy(eu + 0.0).to(TYPES[kind]))


@pytest.mark.gpu
def test_gradient_against_differences():
    """The gradient of sum(dy * y) along changes of the gate's and the other projection's weights, in float32."""
    m, n, k = 70, 50, 200
    gen = torch.Generator().manual_seed(8)
    x, g, u = (torch.randn(r, k, generator=gen) for r in (m, n, n))
    dy = torch.randn(m, n, generator=gen)
    X, G, U = (ifx.fp8_quantize(t.cuda()) for t in (x, g / 8, u / 8))
    xv, gv, uv = (f64(ifx.fp8_dequantize(t, torch.float32)) for t in (X, G, U))
    for act in (0, 2):
        dgate, dup = (f64(t) for t in ifx.gated_backward(dy.cuda(), X, G, U, act))
        def loss(gv, uv):
            return (f64(dy) * lowp.act(xv @ gv.T, act) * (xv @ uv.T)).sum()
        for seed in range(3):
            rng = np.random.default_rng(seed)
            a, b = rng.standard_normal(gv.shape), rng.standard_normal(uv.shape)
            h = 1e-6
            slope = (loss(gv + h * a, uv + h * b) - loss(gv - h * a, uv - h * b)) / (2 * h)
            mine = ((dgate.T @ xv) * a).sum() + ((dup.T @ xv) * b).sum()
            size = (np.abs(dgate.T) @ np.abs(xv) * np.abs(a)).sum() + (np.abs(dup.T) @ np.abs(xv) * np.abs(b)).sum()
            # float32 results: a few roundings of terms; differences in 64 bits: h^2 and 2^-53 / h
            assert abs(slope - mine) <= 2.0 ** -18 * size


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(3, 50), (200, 131), (300, 256)])
def test_pitches_in_place_and_stream(m, n):
    """Results in slices at odd offsets, the gradient over dy itself, another stream: nothing outside is written."""
    k = 260
    q, rng = gated_case(m, n, k, 5)
    X, G, U = (tensor_of(t, k) for t in q)
    s = torch.cuda.Stream()
    for kind in ("bf16", "f32"):
        note(f"gated into slices, {m} x {n} {kind}")
        expect = ifx.gated(X, G, U, 2, TYPES[kind])
        dy = torch.from_numpy(rng.standard_normal((m, n))).to(TYPES[kind]).cuda()
        eg, eu = ifx.gated_backward(dy, X, G, U)
        wide = [torch.full((m, n + 7 + i), 3.0, dtype=TYPES[kind], device="cuda") for i in range(3)]
        y, dg, du = (t[:, 1 + i:1 + i + n] for i, t in enumerate(wide))
        dg.copy_(dy)
        s.wait_stream(torch.cuda.current_stream())
        assert ifx.gated(X, G, U, 2, out=y, stream=s) is y
        ifx.gated_backward(dg, X, G, U, out=(dg, du), stream=s.cuda_stream)
        s.synchronize()
        assert torch.equal(y, expect) and torch.equal(dg, eg) and torch.equal(du, eu)
        for i, t in enumerate(wide):
            assert (t[:, :1 + i] == 3).all() and (t[:, 1 + i + n:] == 3).all()
        du.copy_(dy)
        ifx.gated_backward(du, X, G, U, out=(dg, du))
        assert torch.equal(dg, eg) and torch.equal(du, eu)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [2, 300])
def test_nan_blocks(m):
    """A NaN in a row of X spoils that row alone, one in a weight its column, and so its block of codes."""
    n, k = 300, 200
    q, _ = gated_case(m, n, k, 6)
    q[0][1][0, 1, 1] = 255
    q[1][1][0, 5, 0] = 255
    q[2][0][0, 200, 3] = 0x7f
    X, G, U = (tensor_of(t, k) for t in q)
    y = ifx.gated(X, G, U)
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[1] = nan[:, 5] = nan[:, 200] = True
    assert torch.equal(y.isnan(), nan)
    got = ifx.gated_fp8(X, G, U)
    v = ifx.fp8_dequantize(got, torch.float32).isnan()
    assert bool(v[:, :256].all()) and not v[0, 256:].any() and bool(v[1].all())
    dgate, dup = ifx.gated_backward(torch.ones_like(y), X, G, U)
    assert torch.equal(dgate.isnan(), nan)
    nan[:, 200] = False
    nan[1] = True
    assert torch.equal(dup.isnan(), nan)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("m", [2, 40, 300])
def test_nan_blocks_of_the_gate(m, act):
    """A NaN at the gate reaches the gate's gradient whatever the activation, also where the other projection is finite;
    one at the other projection leaves the other's gradient as it is."""
    n, k = 300, 200
    note(f"NaN at the gate, {m} rows, {act}")
    q, _ = gated_case(m, n, k, 7)
    q[0][1][0, 1, 1] = 255
    q[1][1][0, 5, 0] = 255
    q[1][0][1, 290, 4] = 0xff
    q[2][0][0, 200, 3] = 0x7f
    X, G, U = (tensor_of(t, k) for t in q)
    for kind in ("bf16", "f32"):
        dy = torch.ones(m, n, dtype=TYPES[kind], device="cuda")
        dgate, dup = ifx.gated_backward(dy, X, G, U, ACTS[act])
        at_gate, at_up = (torch.zeros(m, n, dtype=torch.bool, device="cuda") for _ in range(2))
        at_gate[1] = at_up[1] = at_gate[:, 5] = at_gate[:, 290] = at_up[:, 200] = True
        # dgate = dy up act'(gate), dup = dy act(gate); without an activation act' is 1 whatever the gate
        assert torch.equal(dgate.isnan(), at_up if act == "none" else at_gate | at_up)
        assert torch.equal(dup.isnan(), at_gate)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [2, 130])
def test_in_a_graph(m):
    n, k = 260, 700
    q, _ = gated_case(m, n, k, 9)
    X, G, U = (tensor_of(t, k) for t in q)
    dy = torch.randn(m, n, device="cuda").to(torch.bfloat16)
    y, out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), ifx.fp8_empty(m, n)
    grads = (torch.empty_like(dy), torch.empty_like(dy))
    x = torch.randn(m, k, device="cuda")
    ifx.fp8_quantize(x, out=X)
    first = [ifx.gated(X, G, U), ifx.gated_fp8(X, G, U), ifx.gated_backward(dy, X, G, U)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ifx.fp8_quantize(x, out=X)
        ifx.gated(X, G, U, out=y)
        ifx.gated_fp8(X, G, U, out=out)
        ifx.gated_backward(dy, X, G, U, out=grads)
    for i in range(4):
        for t in (y, out.codes, *grads):
            t.zero_()
        x.add_(0.0 if i < 2 else 1.0)
        g.replay()
        Q = ifx.fp8_quantize(x)
        expect = [ifx.gated(Q, G, U), ifx.gated_fp8(Q, G, U), ifx.gated_backward(dy, Q, G, U)]
        torch.cuda.synchronize()
        for e in (expect, first) if i < 2 else (expect,):
            assert torch.equal(y, e[0]) and torch.equal(out.codes, e[1].codes) and torch.equal(out.scales, e[1].scales)
            assert torch.equal(grads[0], e[2][0]) and torch.equal(grads[1], e[2][1])


@pytest.mark.gpu
def test_empty_and_refusals():
    w, x = ifx.fp8_quantize(torch.ones(6, 64, device="cuda")), ifx.fp8_quantize(torch.empty(0, 64, device="cuda"))
    assert ifx.gated(x, w, w).shape == (0, 6) and ifx.gated(w, x, x).shape == (6, 0)
    assert ifx.gated_fp8(x, w, w).codes.shape == (1, 0, 128)
    dgate, dup = ifx.gated_backward(torch.empty(0, 6, device="cuda"), x, w, w)
    assert dgate.shape == dup.shape == (0, 6)
    with pytest.raises(ifx.IfxError):
        ifx.gated(w, w, w, act=9)
    assert ifx.gated_fp8(w, x, x).codes.shape == (0, 6, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,act", [("bf16", "silu"), ("f16", "none"), ("f16", "silu"), ("f32", "silu")])
@pytest.mark.parametrize("extra", [0, 64, 3])
def test_many_large_tiles(kind, act, extra):
    """Large tiles whose ring is refilled many times for both weights, three words of scales, whole tiles and edges inside
    one, results past the caches' size in rows that fill 128-byte lines (extra 0 and 64) and rows that share them.  Every
    result is checked, and what lies beside the rows."""
    m, n, k = 4200, 2112, 1200
    note(f"gated, large tiles {m} x {n} x {k} {kind} {act}, rows of {n + extra}")
    q, _ = gated_case(m, n, k, 31)
    X, G, U = (tensor_of(t, k) for t in q)
    x, gv, uv = (cuda64(t, k) for t in q)
    b = sum_bound(k, kind)
    g, u, tg, tu = x @ gv.t(), x @ uv.t(), b * (x.abs() @ gv.abs().t()), b * (x.abs() @ uv.abs().t())
    s = torch.sigmoid(g)
    a, slope = (g * s, s + g * s * (1 - s)) if act == "silu" else (g, torch.ones_like(g))
    more = (g.abs() + 4) * 2.0 ** -22 if act == "silu" else torch.zeros_like(g)
    y = a * u
    tol = a.abs() * tu + 1.1 * tg * (u.abs() + tu) + (2.0 ** -23 + more) * y.abs()

    def results():
        return torch.full((m, n + extra), 3.0, dtype=TYPES[kind], device="cuda")
    out = results()
    ifx.gated(X, G, U, ACTS[act], out=out[:, :n])
    assert float(y.abs().max()) < 30000 and whole_excess(out[:, :n], y, tol, kind) == 0 and bool((out[:, n:] == 3).all())
    if extra == 0 and kind == "bf16":
        check_fp8(ifx.gated_fp8(X, G, U, ACTS[act]), f64(y), f64(tol), n)
    d = torch.randn(m, n, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(TYPES[kind])
    dg, du = results(), results()
    ifx.gated_backward(d, X, G, U, ACTS[act], out=(dg[:, :n], du[:, :n]))
    d = d.double()
    tol_g = d.abs() * (1.1 * tu + 0.5 * tg * (u.abs() + tu) + (1.1 * more + 2.0 ** -22) * (u.abs() + tu))
    tol_u = d.abs() * (1.1 * tg + (more + 2.0 ** -22) * a.abs())
    assert whole_excess(dg[:, :n], d * u * slope, tol_g, kind) == 0
    assert whole_excess(du[:, :n], d * a, tol_u, kind) == 0
    assert bool((dg[:, n:] == 3).all()) and bool((du[:, n:] == 3).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n,k", [(300, 700), (1000, 5000)])
def test_codes_of_a_row_alone_and_in_a_batch(n, k):
    """Rows of a batch of 17, and each alone, among three and among 16 of them, where other kernels run: sums differ by
    their bounds only."""
    note(f"gated to codes, {n} x {k}")
    q, _ = gated_case(17, n, k, 41)
    X, G, U = (tensor_of(t, k) for t in q)
    y, _, _, tol, _, _ = bounds(q, k, 2, "bf16")
    for rows in [slice(0, 17), slice(0, 16), slice(2, 5)] + [slice(i, i + 1) for i in (0, 7, 16)]:
        part = ifx.Fp8(X.codes[:, rows].contiguous(), X.scales[:, rows].contiguous(), k)
        check_fp8(ifx.gated_fp8(part, G, U), y[rows], tol[rows], n)
