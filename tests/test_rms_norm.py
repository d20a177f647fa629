"""Root mean square norm with the residual's addition, its 8-bit form and its gradient: refusals (CPU) and the kernels
against the 64-bit reference (GPU).

Bounds.  A row's sum of squares is a chain of at most 24 fused additions a thread (three vectors of eight), 6 joins in a
wave and 16 across waves, each off by at most 2^-24 of the sum, so rstd is off by at most 23 2^-24 of itself for the sum and
4 roundings for the rest: 2^-19.  y = h rstd weight adds two roundings: 2^-18 of itself in all, then one rounding to the
type.  The gradient's mean is a chain of as many additions of terms of three roundings: at most 50 2^-24 mean |d xhat|.
dweight's column is a chain over a workgroup's rows (at most ceil(rows / 256) of them and 16 subgroups), 16 joins a lane and
32 across: n = rows / 256 + 66 additions of terms of two roundings, off by at most (n + 2) 2^-24 of the terms' magnitudes.
"""
import ctypes

import numpy as np
import pytest
import torch

import convolution_int8_implicit_amd as ifx
from oracle import lowp
from test_gated import check_fp8
from test_mx4 import TYPES, excess, f64, note

REL = 2.0 ** -18


# ------------------------------------------------------------------------------------------ CPU

def test_reference_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, dy, dh = rng.standard_normal((3, 4, 9))
    w = rng.standard_normal(9)
    def loss(h, w):
        return (dy * lowp.rms_norm(h, w, 1e-3)[0]).sum() + (dh * h).sum()
    dx, dw = lowp.rms_norm_backward(dy, h, lowp.rms_norm(h, w, 1e-3)[1], w, dh)
    for _ in range(3):
        a, b = rng.standard_normal((4, 9)), rng.standard_normal(9)
        e = 1e-6
        slope = (loss(h + e * a, w + e * b) - loss(h - e * a, w - e * b)) / (2 * e)
        assert abs(slope - ((dx * a).sum() + (dw * b).sum())) < 1e-7


def test_refusals_need_no_device():
    L = ifx.lib()
    fake, odd, half = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001), ctypes.c_void_p(0x100002)

    def desc(rows=4, c=5, t=1, eps=1e-5, ld_x=5, ld_res=5, ld_h=5, ld_y=5, ld_dy=5, ld_dh=5):
        return ctypes.byref(ifx.RmsDesc(rows, c, t, eps, ld_x, ld_res, ld_h, ld_y, ld_dy, ld_dh))

    def typed(x=fake, res=fake, w=fake, h=fake, y=fake, rstd=fake, **kw):
        return L.ifx_rms_norm(desc(**kw), x, res, w, h, y, rstd, None)

    def eight(x=fake, res=fake, w=fake, h=fake, codes=fake, scales=fake, rstd=fake, **kw):
        return L.ifx_rms_norm_fp8(desc(**kw), x, res, w, h, codes, scales, rstd, None)

    def backward(dy=fake, x=fake, rstd=fake, w=fake, dh=fake, dx=fake, dw=fake, ws=fake, ws_bytes=1 << 30, **kw):
        return L.ifx_rms_norm_backward(desc(**kw), dy, x, rstd, w, dh, dx, dw, ws, ws_bytes, None)
    assert L.ifx_rms_norm(None, *[fake] * 6, None) == 1 and L.ifx_rms_norm_fp8(None, *[fake] * 7, None) == 1
    assert L.ifx_rms_norm_backward(None, *[fake] * 8, 0, None) == 1 and L.ifx_rms_norm_workspace_bytes(None) == 0
    for call in (typed, eight, backward):
        assert call(t=3) == 3 and call(c=24577, ld_x=1 << 15) == 3
        assert call(rows=-1) == 2 and call(c=0) == 2 and call(eps=-1.0) == 2 and call(eps=float("nan")) == 2
        assert call(ld_x=4) == 2 and call(ld_x=1 << 61) == 2
        assert call(rows=1 << 23, c=8193, ld_x=8193) == 2  # more work-items than a launch holds
        assert call(x=None) == 1 and call(x=odd) == 4 and call(rstd=half) == 4 and call(w=half) == 4
    for call in (typed, eight):
        assert call(ld_res=4) == 2 and call(ld_h=4) == 2 and call(res=odd) == 4 and call(h=odd) == 4
        assert call(rows=0, x=None) == 0
    assert typed(y=None) == 1 and typed(ld_y=4) == 2 and typed(y=odd) == 4
    assert eight(codes=None) == 1 and eight(scales=None) == 1 and eight(codes=half) == 4
    # absent operands' pitches are not looked at
    assert typed(res=None, ld_res=0, h=None, ld_h=0, y=None) == 1 and eight(res=None, ld_res=0, ld_y=0, codes=None) == 1
    for name in ("dy", "rstd", "dx"):
        assert backward(**{name: None}) == 1
    assert backward(dy=odd) == 4 and backward(dx=odd) == 4 and backward(dh=odd) == 4 and backward(dw=half) == 4
    assert backward(ld_dy=4) == 2 and backward(ld_y=4) == 2 and backward(ld_dh=4) == 2
    need = L.ifx_rms_norm_workspace_bytes(desc(rows=300))
    assert need >= 5 * 4 and L.ifx_rms_norm_workspace_bytes(desc(rows=0)) == 0
    assert backward(rows=300, ws_bytes=need - 1) == 5 and backward(rows=300, ws=None) == 1 and backward(rows=300, ws=half) == 4
    assert L.ifx_rms_norm_workspace_bytes(desc(rows=1 << 20, c=8192, ld_x=8192)) == 512 * 8192 * 4
    assert backward(rows=0, dw=None, dy=None) == 0


def test_binding_refusals_need_no_device(monkeypatch):
    with pytest.raises(ValueError):
        ifx.rms_norm(torch.zeros(4, 32))  # not on a GPU
    monkeypatch.setattr(ifx, "_on_device", lambda *ts: 0)
    monkeypatch.setattr(ifx, "_raw_stream", lambda stream, index: 0)

    def t(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="meta")
    x = t(4, 32)
    for call in (ifx.rms_norm, ifx.rms_norm_fp8):
        for kw in (dict(weight=t(31)), dict(weight=t(32, dtype=torch.bfloat16)), dict(residual=t(4, 31)),
                   dict(residual=t(4, 32, dtype=torch.float16)), dict(sum_out=t(32, 4))):
            with pytest.raises(ValueError):
                call(x, **kw)
        with pytest.raises(TypeError):
            call(t(4, 32, dtype=torch.int8))
        with pytest.raises(ValueError):
            call(t(32, 4).t())
        with pytest.raises(ValueError, match="32 bits"):
            call(t((1 << 32) + 5, 3))
    with pytest.raises(ValueError):
        ifx.rms_norm(x, out=t(4, 33))
    with pytest.raises(ValueError):
        ifx.rms_norm_fp8(x, out=ifx.fp8_empty(4, 33, device="meta"))
    for args in ((t(4, 31), x, t(4)), (x, x, t(5)), (x, x, t(4, dtype=torch.float16))):
        with pytest.raises(ValueError):
            ifx.rms_norm_backward(*args)
    with pytest.raises(ValueError):
        ifx.rms_norm_backward(x, x, t(4), dh=t(5, 32))
    with pytest.raises(ValueError):
        ifx.rms_norm_backward(x, x, t(4), out=t(4, 32, dtype=torch.bfloat16))


class Recorded:
    """Stands in for the library: keeps the arguments of the last call."""

    def ifx_rms_norm(self, d, x, res, weight, h, y, rstd, stream):
        self.h, self.y, self.ld_h, self.ld_y = h, y, d.ld_h, d.ld_y
        return 0


def test_shared_memory_needs_no_device(monkeypatch):
    """Without a residual the sum is x itself, but not where out takes x's place: then it is memory of its own.  out and
    sum_out may not share memory."""
    monkeypatch.setattr(ifx, "_on_device", lambda *ts: 0)
    monkeypatch.setattr(ifx, "_raw_stream", lambda stream, index: 0)
    rec = Recorded()
    monkeypatch.setattr(ifx, "lib", lambda: rec)
    wide = torch.zeros(4, 80)
    for x in (torch.zeros(4, 32), wide[:, 3:35], wide.view(2, 2, 80)[..., 1:33]):
        y, h, _ = ifx.rms_norm(x)
        assert h is x and rec.h is None
        y, h, _ = ifx.rms_norm(x, out=torch.zeros_like(x))
        assert h is x and rec.h is None
        y, h, _ = ifx.rms_norm(x, out=x)
        assert y is x and rec.y == x.data_ptr() and rec.ld_y == ifx._pitch(x)[2]
        assert h.shape == x.shape and rec.h == h.data_ptr() != x.data_ptr() and rec.ld_h == 32
        y, h, _ = ifx.rms_norm(x, residual=torch.zeros_like(x), out=x)
        assert y is x and h is not x and rec.h == h.data_ptr()
        for kw in (dict(out=x, sum_out=x), dict(out=x, sum_out=x, residual=torch.zeros_like(x))):
            with pytest.raises(ValueError, match="share"):
                ifx.rms_norm(x, **kw)
        y, h, _ = ifx.rms_norm(x, out=torch.zeros_like(x), sum_out=x)
        assert h is x and rec.h == x.data_ptr()
    # side by side in wider rows they share nothing, one element further they do
    ifx.rms_norm(torch.zeros(4, 32), out=wide[:, 3:35], sum_out=wide[:, 35:67])
    ifx.rms_norm(torch.zeros(4, 32), out=wide[:, 48:], sum_out=wide[:, 16:48])
    for a, b in ((3, 34), (34, 3), (48, 17)):
        with pytest.raises(ValueError, match="share"):
            ifx.rms_norm(torch.zeros(4, 32), out=wide[:, a:a + 32], sum_out=wide[:, b:b + 32])
    flat = torch.zeros(256)
    ifx.rms_norm(torch.zeros(4, 32), out=flat[:128].view(4, 32), sum_out=flat[128:].view(4, 32))
    with pytest.raises(ValueError, match="share"):
        ifx.rms_norm(torch.zeros(4, 32), out=flat[:128].view(4, 32), sum_out=flat[127:255].view(4, 32))
    none = torch.zeros(0, 32)
    ifx.rms_norm(none, out=none, sum_out=none)


# ------------------------------------------------------------------------------------------ GPU

# every row width at the edges of the kernels' ranges, many rows and few, rows inside a workgroup's group
SHAPES = [(1, 1), (3, 7), (5, 8), (17, 9), (33, 127), (16, 128), (40, 129), (9, 511), (7, 512), (600, 513), (5, 1000), (700, 1024),
          (3, 1025), (520, 2047), (6, 2048), (530, 2049), (5, 4096), (515, 4099), (4, 8192), (520, 8190), (2, 8193), (3, 16384),
          (3, 16385), (2, 24576), (2, 24571)]


def rms_case(rows, c, kind, seed):
    rng = np.random.default_rng(seed)
    x, r, dy, dh = (torch.from_numpy(rng.standard_normal((rows, c)) * s).to(TYPES[kind])
                    for s in (np.exp(0.5 * rng.standard_normal(c)), 2.0, 1.0, 1.0))
    return x, r, dy, dh, torch.from_numpy(1 + 0.3 * rng.standard_normal(c)).float()


def check_rms(y, h, rstd, weight, eps, kind):
    exact, er = lowp.rms_norm(f64(h), None if weight is None else f64(weight), eps)
    assert (np.abs(f64(rstd) - er) <= 2.0 ** -19 * er).all()
    assert excess(f64(y), exact, REL * np.abs(exact), kind) == 0


def check_grad(dx, dw, dy, h, rstd, w, dh, kind):
    d64, h64, r64 = f64(dy), f64(h), f64(rstd)
    w64 = np.ones(h64.shape[1]) if w is None else f64(w)
    ex, ew = lowp.rms_norm_backward(d64, h64, r64, w64, None if dh is None else f64(dh))
    xhat = np.abs(h64 * r64[:, None])
    d = np.abs(d64 * w64)
    m = (d * xhat).mean(-1, keepdims=True)
    tol = r64[:, None] * (xhat * m * (50 + 4) + 4 * d) * 2.0 ** -24
    if dh is not None:
        tol = tol + (np.abs(f64(dh)) + np.abs(ex)) * 2.0 ** -23
    assert excess(f64(dx), ex, tol, kind) == 0
    n = h64.shape[0] // 256 + 66
    assert (np.abs(f64(dw) - ew) <= (n + 2) * 2.0 ** -24 * np.abs(d64 * xhat).sum(0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,c", SHAPES)
def test_norm_and_gradient(rows, c):
    for i, kind in enumerate(("f32", "bf16", "f16")):
        note(f"rms norm {rows} x {c} {kind}")
        x, r, dy, dh, w = rms_case(rows, c, kind, 10 * rows + c + i)
        X, R, W = x.cuda(), r.cuda(), w.cuda()
        # with the residual: the sum is rounded to the type, the norm is that of the rounded sum
        y, h, rstd = ifx.rms_norm(X, W, R)
        assert torch.equal(h.cpu(), (x.float() + r.float()).to(TYPES[kind])) and rstd.shape == (rows,)
        check_rms(y, h, rstd, w, 1e-5, kind)
        q, h2, rstd2 = ifx.rms_norm_fp8(X, W, R)
        assert torch.equal(h, h2) and torch.equal(rstd, rstd2)
        exact, _ = lowp.rms_norm(f64(h), f64(w), 1e-5)
        check_fp8(q, exact, REL * np.abs(exact), c)
        # without residual and weight
        y, h, rstd = ifx.rms_norm(X, eps=0.5)
        assert h is X
        check_rms(y, x, rstd, None, 0.5, kind)
        for W1, dh1 in ((W, dh.cuda()), (W, None), (None, None)):
            dx, dw = ifx.rms_norm_backward(dy.cuda(), X, rstd, W1, dh1)
            check_grad(dx, dw, dy, x, rstd, W1, None if dh1 is None else dh, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,c,kind", [(5000, 510, "f16"), (40000, 100, "bf16"), (4111, 1000, "f32"), (3001, 4096, "bf16"),
                                         (1100, 8192, "f32"), (2100, 6001, "f16"), (1050, 9000, "bf16"), (1030, 20000, "bf16")])
def test_many_rows(rows, c, kind):
    """Workgroups that take several rows in turn, results past the caches' size among them."""
    note(f"rms norm {rows} x {c} {kind}")
    x, r, dy, dh, w = rms_case(rows, c, kind, rows)
    y, h, rstd = ifx.rms_norm(x.cuda(), w.cuda(), r.cuda())
    check_rms(y, h, rstd, w, 1e-5, kind)
    dx, dw = ifx.rms_norm_backward(dy.cuda(), h, rstd, w.cuda(), dh.cuda())
    check_grad(dx, dw, dy, h, rstd, w, dh, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,c,off", [(3, 50, 1), (37, 1000, 3), (520, 4096, 8)])
def test_pitches_in_place_and_stream(rows, c, off):
    """Operands and results in slices at odd offsets, the sum over the residual, y over x, dx over each of its operands,
    another stream: nothing outside the slices is written, and the results are those of plain tensors."""
    s = torch.cuda.Stream()
    for kind in ("bf16", "f32"):
        note(f"rms norm in slices, {rows} x {c} {kind}")
        x, r, dy, dh, w = (t.cuda() for t in rms_case(rows, c, kind, 5))
        y, h, rstd = ifx.rms_norm(x, w, r)
        q, _, _ = ifx.rms_norm_fp8(x, w, r)
        dx, dw = ifx.rms_norm_backward(dy, h, rstd, w, dh)

        def slices(*ts):
            wide = [torch.full((rows, c + 2 * off + 5 + i), 3.0, dtype=TYPES[kind], device="cuda") for i in range(len(ts))]
            inner = [t[:, off:off + c] for t in wide]
            for i, t in zip(inner, ts):
                i.copy_(t)
            s.wait_stream(torch.cuda.current_stream())
            return wide, inner

        def clean(wide):
            return all(bool((t[:, :off] == 3).all()) and bool((t[:, off + c:] == 3).all()) for t in wide)
        wide, (x1, r1) = slices(x, r)
        y1, h1, rstd1 = ifx.rms_norm(x1, w, r1, out=x1, sum_out=r1, stream=s)
        s.synchronize()
        assert y1 is x1 and h1 is r1 and torch.equal(x1, y) and torch.equal(r1, h) and torch.equal(rstd1, rstd) and clean(wide)
        wide, (x1, r1) = slices(x, r)
        q1, h1, _ = ifx.rms_norm_fp8(x1, w, r1, sum_out=x1, stream=s.cuda_stream)
        s.synchronize()
        assert torch.equal(q1.codes, q.codes) and torch.equal(q1.scales, q.scales) and torch.equal(x1, h) and clean(wide)
        for target in range(3):
            wide, (dy1, h1, dh1) = slices(dy, h, dh)
            out = (dy1, h1, dh1)[target]
            dx1, dw1 = ifx.rms_norm_backward(dy1, h1, rstd, w, dh1, out=out, stream=s)
            s.synchronize()
            assert dx1 is out and torch.equal(out, dx) and torch.equal(dw1, dw) and clean(wide)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,c", [(3, 50), (520, 4096), (5, 20000)])
def test_in_place_without_a_residual(rows, c):
    """y over x: the sum that comes back is still x, and its gradient that of plain tensors."""
    for kind in ("bf16", "f32"):
        note(f"rms norm over its input, {rows} x {c} {kind}")
        x, _, dy, dh, w = (t.cuda() for t in rms_case(rows, c, kind, 6))
        y, _, rstd = ifx.rms_norm(x, w)
        dx, dw = ifx.rms_norm_backward(dy, x, rstd, w, dh)
        wide = torch.full((rows, c + 9), 3.0, dtype=TYPES[kind], device="cuda")
        x1 = wide[:, 4:4 + c]
        x1.copy_(x)
        y1, h1, rstd1 = ifx.rms_norm(x1, w, out=x1)
        assert y1 is x1 and torch.equal(x1, y) and torch.equal(h1, x) and torch.equal(rstd1, rstd)
        assert (wide[:, :4] == 3).all() and (wide[:, 4 + c:] == 3).all()
        dx1, dw1 = ifx.rms_norm_backward(dy, h1, rstd1, w, dh)
        assert torch.equal(dx1, dx) and torch.equal(dw1, dw)


@pytest.mark.gpu
@pytest.mark.parametrize("c", [100, 1000, 3000, 9000])
def test_extreme_rows(c):
    """Rows of zeros, rows whose squares overflow or vanish, infinities and NaN: each spoils its own row alone."""
    note(f"extreme rows of {c}")
    x = torch.ones(8, c)
    x[1] = 0
    x[2] = 3e38
    x[3] = 1e30 * torch.linspace(-1, 1, c)
    x[4, c // 2] = float("nan")
    x[5, c - 1] = float("inf")
    x[6] = 1e-30
    for kind in ("f32", "bf16"):
        X = x.to(TYPES[kind])
        y, _, rstd = ifx.rms_norm(X.cuda())
        keep = [0, 1, 2, 3, 6, 7]
        check_rms(y[keep], X[keep], rstd[keep], None, 1e-5, kind)
        assert y[4].isnan().all() and torch.isnan(rstd[4])
        # rstd is 0: finite values give 0, the infinity a NaN
        assert rstd[5] == 0 and y[5, c - 1].isnan() and not y[5, :c - 1].any()
        q, _, _ = ifx.rms_norm_fp8(X.cuda())
        v = ifx.fp8_dequantize(q, torch.float32)
        assert v[4].isnan().all() and not v[keep].isnan().any() and not v[1].any()
        assert v[5, (c - 1) // 128 * 128:].isnan().all() and not v[5, :(c - 1) // 128 * 128].any()
    big = torch.full((2, c), 60000.0, dtype=torch.float16)
    y, h, rstd = ifx.rms_norm(big.cuda(), residual=-big.cuda())
    assert not y.any() and not h.any()
    y, h, rstd = ifx.rms_norm(big.cuda(), residual=big.cuda())  # the sum overflows float16
    assert h.isinf().all() and y.isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("c", [100, 1000, 3000, 20000])
def test_rows_past_the_largest_square_with_a_large_eps(c):
    """eps counts also in a row whose squares overflow."""
    x = torch.zeros(3, c)
    x[:, c // 3] = torch.tensor([2e19, -3e20, 1e10])
    for eps in (1e34, 3e36, 3e38):
        note(f"rows of {c}, eps {eps}")
        y, _, rstd = ifx.rms_norm(x.cuda(), eps=eps)
        eps32 = float(np.float32(eps))
        check_rms(y, x, rstd, None, eps32, "f32")


@pytest.mark.gpu
def test_empty():
    w = torch.ones(40, device="cuda")
    none = torch.empty(0, 40, device="cuda", dtype=torch.bfloat16)
    y, h, rstd = ifx.rms_norm(none, w, none)
    assert y.shape == h.shape == (0, 40) and rstd.shape == (0,)
    q, _, _ = ifx.rms_norm_fp8(none, w)
    assert q.codes.shape == (1, 0, 128)
    dx, dw = ifx.rms_norm_backward(none, none, rstd, w)
    assert dx.shape == (0, 40) and dw.shape == (40,) and not dw.any()
    with pytest.raises(ifx.IfxError):
        ifx.rms_norm(torch.zeros(2, 24577, device="cuda"))
    with pytest.raises(ifx.IfxError):
        ifx.rms_norm(torch.zeros(2, 0, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,c", [(3, 2048), (2000, 700)])
def test_in_a_graph(rows, c):
    x, r, dy, dh, w = (t.cuda() for t in rms_case(rows, c, "bf16", 3))
    y, h, q, dx = torch.empty_like(x), torch.empty_like(x), ifx.fp8_empty(rows, c), torch.empty_like(x)

    def calls(**kw):
        a = ifx.rms_norm(x, w, r, out=kw.get("y"), sum_out=kw.get("h"))
        b = ifx.rms_norm_fp8(x, w, r, out=kw.get("q"))
        return a, b, ifx.rms_norm_backward(dy, a[1], a[2], w, dh, out=kw.get("dx"))
    first = calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, _, (_, dw) = calls(y=y, h=h, q=q, dx=dx)
    for i in range(4):
        for t in (y, h, q.codes, dx, dw):
            t.zero_()
        x.add_(0.0 if i < 2 else 1.0)
        g.replay()
        expect = calls()
        torch.cuda.synchronize()
        for a, b, d in (expect, first) if i < 2 else (expect,):
            assert torch.equal(y, a[0]) and torch.equal(h, a[1]) and torch.equal(q.codes, b[0].codes)
            assert torch.equal(q.scales, b[0].scales) and torch.equal(dx, d[0]) and torch.equal(dw, d[1])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows past 2^31 elements and 2^32 bytes, in more axes than two."""
    rows, c = (1 << 21) + 7, 1040
    note(f"rms norm {rows} x {c}")
    x = torch.zeros(1, rows, c, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(37, c, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[0, -37:] = tail
    y, h, rstd = ifx.rms_norm(x)
    check_rms(y[0, -37:], x[0, -37:], rstd[-37:], None, 1e-5, "bf16")
    assert not y[0, :-37].any()
    del y
    q, _, _ = ifx.rms_norm_fp8(x)
    exact, _ = lowp.rms_norm(f64(x[0, -37:]), None, 1e-5)
    check_fp8(ifx.Fp8(q.codes[:, -37:], q.scales[:, -37:], c), exact, REL * np.abs(exact), c)
    assert not q.codes[:, :-37].any()
    del q
    dx, dw = ifx.rms_norm_backward(x, x, rstd)
    check_grad(dx[0, -37:], dw, x[0, -37:], x[0, -37:], rstd[-37:], None, None, "bf16")
    assert not dx[0, :-37].any()
