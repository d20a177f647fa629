"""Group norm with an activation, its gradient and its 4-bit form: the 64-bit reference's own pins and the entry
points' refusals (CPU), and the kernels against the reference (GPU).

Bounds, with e = 2^-24 and every 32-bit sum taken in partial sums of a few dozen terms joined pairwise or in
a few dozen steps, so off by at most 64 e times the sum of its terms' magnitudes:
  mean   64 e mean|x|
  rstd   relative 40 e + 2 rstd^2 (mean's error)^2     (half of the variance's 64 e, a root and a division)
  z      |w| (rstd d(mean) + |xhat| d(rstd)/rstd) + 4 e (|w xhat| + |w rstd mean| 2 + |b|)
  act    ReLU keeps an error, SiLU stretches it by at most 1.1 and adds (|z| + 4) 4 e |y|
  output one rounding to its type
The gradient takes mean and rstd as given.  e_xhat = 3 e |xhat|; e_z = |w| e_xhat + 2 e (|w xhat| + |z|);
e_dz = |dy| (0.55 e_z + (|z| + 8) 2 e) for SiLU, 2 e |dy| otherwise (a ReLU's corner is decided by z in
single 32-bit operations, as here); sums as above on top of their terms' own errors.
"""
import ctypes
import os
import random
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import convolution_int8_implicit_amd as ifx
from oracle import lowp

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = 2.0 ** -149  # the smallest float32
E = 2.0 ** -24


def note(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def excess(got, exact, tol, kind):
    """How far `got`, of the type `kind`, lies outside what the values exact - tol .. exact + tol round to (0:
    within): rounding keeps order, so a right result lies between the two ends' roundings."""
    low, high = (f64(torch.from_numpy(exact + s * tol).to(TYPES[kind])) for s in (-1, 1))
    out = np.maximum(np.maximum(low - got, got - high), 0)
    out = np.where(np.isnan(exact) & np.isnan(got), 0.0, out)
    return float(np.max(out)) if out.size and not np.isnan(out).any() else (0.0 if not out.size else np.inf)


def case(n, hw, c, kind, seed):
    """x with channels of their own means and spreads, dy, weight, bias."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, hw, c)) * np.exp(0.5 * rng.standard_normal(c)) + 2 * rng.standard_normal(c)
    x = torch.from_numpy(x).to(TYPES[kind])
    dy = torch.from_numpy(rng.standard_normal((n, hw, c))).to(TYPES[kind])
    w = torch.from_numpy(1 + 0.5 * rng.standard_normal(c)).float()
    b = torch.from_numpy(0.5 * rng.standard_normal(c)).float()
    return x, dy, w, b


def group_mean(v, groups):
    return lowp._by_group(v, groups).mean(-1)


def forward_bounds(x, groups, w, b, eps):
    c = x.shape[2]
    z, xhat, mean, rstd = lowp.group_norm(x, groups, w, b, eps)
    dm = 64 * E * group_mean(np.abs(x), groups)
    dr = 40 * E + 2 * (rstd * dm) ** 2
    rs = lowp.spread(rstd, c)
    tz = np.abs(w) * (rs * lowp.spread(dm, c) + np.abs(xhat) * lowp.spread(dr, c))
    tz = tz + 4 * E * (np.abs(w * xhat) + 2 * np.abs(w * rs * lowp.spread(mean, c)) + np.abs(b))
    return z, mean, rstd, tz, dm, dr


def worst(got, expect, tol):
    assert got.shape == expect.shape
    return float(np.max(np.abs(got - expect) / tol)) if got.size else 0.0


def check_forward(x, groups, w, b, eps, act, y, mean, rstd, kind):
    z, em, er, tz, dm, dr = forward_bounds(f64(x), groups, f64(w), f64(b), eps)
    ey = lowp.act(z, act)
    ty = 1.1 * tz + (np.abs(z) + 4) * 4 * E * np.abs(ey) if act == 2 else tz
    assert worst(f64(mean), em, dm + TINY) <= 1
    assert worst(f64(rstd), er, er * dr) <= 1
    assert excess(f64(y), ey, ty, kind) == 0


def z_in_32_bits(x, mean, rstd, w, b):
    c = x.shape[2]
    m, r = (np.repeat(t.cpu().numpy(), c // t.shape[1], axis=1)[:, None, :] for t in (mean, rstd))
    xh = (x.float().cpu().numpy() - m) * r
    return xh * w.cpu().numpy() + b.cpu().numpy()


def check_backward(dy, x, mean, rstd, groups, w, b, act, dx, dw, db, kind):
    n, hw, c = x.shape
    z32 = z_in_32_bits(x, mean, rstd, w, b) if act == 1 else None
    ex, ew, eb, (xhat, z, dz, d) = lowp.group_norm_backward(f64(dy), f64(x), f64(mean), f64(rstd), groups, f64(w),
                                                            f64(b), act, z32)
    a, W = np.abs, np.abs(f64(w))
    exh = 3 * E * a(xhat)
    ez = W * exh + 2 * E * (W * a(xhat) + a(z))
    edz = a(f64(dy)) * ((0.55 * ez + (a(z) + 8) * 2 * E) if act == 2 else 2 * E)
    ed = W * edz + E * a(d)
    r = lowp.spread(f64(rstd), c)
    t1 = group_mean(64 * E * a(d * xhat) + ed * a(xhat) + a(d) * exh, groups)
    t2 = group_mean(64 * E * a(d) + ed, groups)
    m1, m2 = group_mean(d * xhat, groups), group_mean(d, groups)
    s = lowp.spread
    tx = ed + s(t2, c) + a(xhat) * s(t1, c) + exh * a(s(m1, c)) + 4 * E * (a(d) + a(s(m2, c)) + a(xhat * s(m1, c)))
    tx = r * tx + E * a(ex)
    assert excess(f64(dx), ex, tx, kind) == 0
    tw = (64 * E * a(dz * xhat) + edz * a(xhat) + a(dz) * exh).sum((0, 1)) + TINY
    tb = (64 * E * a(dz) + edz).sum((0, 1)) + TINY
    assert worst(f64(dw), ew, tw) <= 1
    assert worst(f64(db), eb, tb) <= 1


# ------------------------------------------------------------------------------------------ CPU

def test_reference_pins():
    """Statistics of a ramp in closed form, and the gradient against differences of the forward pass."""
    x = np.arange(12, dtype=np.float64).reshape(1, 3, 4)
    z, xhat, mean, rstd = lowp.group_norm(x, 2, np.ones(4), np.zeros(4), 0.0)
    assert mean.tolist() == [[4.5, 6.5]] and np.allclose(rstd, 1 / np.sqrt((2 * (16 + 0) + 1.5) / 3), rtol=0.02)
    assert np.allclose(group_mean(xhat, 2), 0) and np.allclose(group_mean(xhat ** 2, 2), 1)
    rng = np.random.default_rng(0)
    for act in (0, 1, 2):
        x, dy, w, b = (rng.standard_normal(s) for s in ((2, 5, 6), (2, 5, 6), 6, 6))

        def loss(x, w, b):
            return (dy * lowp.act(lowp.group_norm(x, 3, w, b, 1e-5)[0], act)).sum()
        _, _, mean, rstd = lowp.group_norm(x, 3, w, b, 1e-5)
        grads = lowp.group_norm_backward(dy, x, mean, rstd, 3, w, b, act)
        for i, (grad, at) in enumerate(zip(grads, (x, w, b))):
            v = rng.standard_normal(at.shape)
            step = [1e-6 * v if j == i else 0 for j in range(3)]
            diff = (loss(x + step[0], w + step[1], b + step[2]) - loss(x - step[0], w - step[1], b - step[2])) / 2e-6
            assert abs(diff - (grad * v).sum()) < 1e-6 * (1 + np.abs(grad * v).sum())


def test_refusals_need_no_device():
    L = ifx.lib()
    fake, odd, half = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001), ctypes.c_void_p(0x100002)

    def desc(n=2, hw=9, c=8, groups=4, t=1, act=0, eps=1e-5, ld_x=8, ld_y=8, ld_dy=8):
        return ifx.GnDesc(n, hw, c, groups, t, act, eps, ld_x, ld_y, ld_dy)

    big = 1 << 40

    def fwd(d, x=fake, w=fake, b=fake, y=fake, m=fake, r=fake, ws=fake, nb=big):
        return L.ifx_group_norm(ctypes.byref(d), x, w, b, y, m, r, ws, nb, None)

    def mx4(d, x=fake, w=fake, b=fake, codes=fake, scales=fake, m=fake, r=fake, ws=fake, nb=big):
        return L.ifx_group_norm_mx4(ctypes.byref(d), x, w, b, codes, scales, m, r, ws, nb, None)

    def bwd(d, dy=fake, x=fake, m=fake, r=fake, w=fake, b=fake, dx=fake, dw=fake, db=fake, ws=fake, nb=big):
        return L.ifx_group_norm_backward(ctypes.byref(d), dy, x, m, r, w, b, dx, dw, db, ws, nb, None)

    for call in (fwd, mx4, bwd):
        for bad in (dict(n=-1), dict(hw=0), dict(c=0), dict(groups=0), dict(groups=3), dict(eps=-1.0),
                    dict(eps=float("nan")), dict(ld_x=7)):
            assert call(desc(**bad)) == 2, (call, bad)
        for bad in (dict(t=3), dict(act=3), dict(c=8200, groups=8, ld_x=8200, ld_y=8200, ld_dy=8200)):
            assert call(desc(**bad)) == 3, (call, bad)
        assert call(desc(), x=None) == 1 and call(desc(), x=odd) == 4
        assert call(desc(), w=half) == 4 and call(desc(), b=half) == 4 and call(desc(), m=half) == 4
        assert call(desc(), ws=ctypes.c_void_p(0x100004)) == 4
    assert fwd(desc(ld_y=7)) == 2 and bwd(desc(ld_y=7)) == 2 and bwd(desc(ld_dy=7)) == 2
    assert fwd(desc(), y=None) == 1 and fwd(desc(), y=odd) == 4
    assert mx4(desc(), codes=None) == 1 and mx4(desc(), scales=None) == 1 and mx4(desc(), codes=half) == 4
    assert bwd(desc(), dy=None) == 1 and bwd(desc(), dx=None) == 1 and bwd(desc(), m=None) == 1
    assert bwd(desc(), dw=half) == 4 and bwd(desc(), dy=odd) == 4
    assert fwd(desc(n=0), x=None, y=None, ws=None, nb=0) == 0 and mx4(desc(n=0), x=None, codes=None) == 0
    assert L.ifx_group_norm(None, fake, fake, fake, fake, fake, fake, fake, big, None) == 1
    # a workspace that is needed is asked for
    d = desc(n=3, hw=100003, c=64, groups=8, ld_x=64, ld_y=64, ld_dy=64)
    for backward, call in ((0, fwd), (0, mx4), (1, bwd)):
        need = L.ifx_group_norm_workspace_bytes(ctypes.byref(d), backward)
        assert need > 0
        assert call(d, nb=need - 1) == 5 and call(d, ws=None, nb=need) == 1
    assert L.ifx_group_norm_workspace_bytes(ctypes.byref(desc(c=9)), 0) == 0


# ------------------------------------------------------------------------------------------ GPU

# single pixels and channels, groups of one channel, of part of a vector, of several, one group of all;
# channel counts around 8, 32 and 128 columns and past 2048; pixels around the batches and chunks
SHAPES = [(1, 1, 1, 1), (2, 1, 32, 8), (1, 7, 8, 8), (3, 49, 20, 4), (2, 100, 24, 8), (2, 65, 60, 12), (1, 784, 128, 32),
          (5, 33, 130, 13), (2, 300, 257, 1), (1, 1517, 64, 16), (70, 9, 96, 32), (1, 20, 2056, 8), (2, 3, 8192, 32),
          (1, 5000, 33, 3), (1, 4099, 512, 32), (2, 12544, 64, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,hw,c,groups", SHAPES)
def test_forward(n, hw, c, groups):
    note(f"group norm {n} x {hw} x {c}, {groups} groups")
    for kind, act in (("f32", 2), ("bf16", 1), ("f16", 0)):
        x, _, w, b = case(n, hw, c, kind, n + hw + c)
        y, mean, rstd = ifx.group_norm(x.cuda(), groups, w.cuda(), b.cuda(), 1e-5, act)
        assert y.dtype == x.dtype and mean.shape == rstd.shape == (n, groups)
        check_forward(x, groups, w, b, 1e-5, act, y, mean, rstd, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("n,hw,c,groups", SHAPES)
def test_backward(n, hw, c, groups):
    note(f"group norm gradient {n} x {hw} x {c}, {groups} groups")
    for kind, act in (("f32", 2), ("bf16", 1), ("f16", 0), ("f32", 1), ("bf16", 2)):
        x, dy, w, b = case(n, hw, c, kind, 2 * n + hw + c)
        _, _, mean, rstd = lowp.group_norm(f64(x), groups, f64(w), f64(b), 1e-5)
        mean, rstd = torch.from_numpy(mean).float(), torch.from_numpy(rstd).float()
        dx, dw, db = ifx.group_norm_backward(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), groups, w.cuda(), b.cuda(), act)
        check_backward(dy, x, mean, rstd, groups, w, b, act, dx, dw, db, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("pitch", [64, 72])
def test_results_larger_than_the_caches(pitch):
    """Two samples of 70000 pixels, 18 MB of bf16, in rows that fill 128-byte lines and rows that share them."""
    n, hw, c, groups = 2, 70000, 64, 8
    x, dy, w, b = case(n, hw, c, "bf16", 91)
    wd, bd = w.cuda(), b.cuda()
    y, dx = (torch.full((n, hw, pitch), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    note(f"group_norm {n}x{hw}x{c} pitch {pitch}")
    _, mean, rstd = ifx.group_norm(x.cuda(), groups, wd, bd, 1e-5, ifx.ACT_SILU, out=y[:, :, :c])
    _, dw, db = ifx.group_norm_backward(dy.cuda(), x.cuda(), mean, rstd, groups, wd, bd, ifx.ACT_SILU, out=dx[:, :, :c])
    check_forward(x, groups, w, b, 1e-5, ifx.ACT_SILU, y[:, :, :c], mean, rstd, "bf16")
    check_backward(dy, x, mean, rstd, groups, w, b, ifx.ACT_SILU, dx[:, :, :c], dw, db, "bf16")
    assert bool((y[:, :, c:] == 7).all()) and bool((dx[:, :, c:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("act", [0, 1, 2])
def test_gradient_against_differences(act):
    """The kernel's gradient along a direction against the difference of the 64-bit forward pass; off by
    the gradient's bounds summed over the direction."""
    n, hw, c, groups = 2, 30, 24, 6
    x, dy, w, b = case(n, hw, c, "f32", 5)
    y, mean, rstd = ifx.group_norm(x.cuda(), groups, w.cuda(), b.cuda(), 1e-5, act)
    grads = ifx.group_norm_backward(dy.cuda(), x.cuda(), mean, rstd, groups, w.cuda(), b.cuda(), act)
    rng = np.random.default_rng(8)
    at = [f64(x), f64(w), f64(b)]

    def loss(at):
        return (f64(dy) * lowp.act(lowp.group_norm(at[0], groups, at[1], at[2], 1e-5)[0], act)).sum()
    for i, grad in enumerate(grads):
        v = rng.standard_normal(at[i].shape)
        h = 1e-6
        up, down = ([t + s * h * v if j == i else t for j, t in enumerate(at)] for s in (1, -1))
        diff = (loss(up) - loss(down)) / (2 * h)
        # 1e-5: mean and rstd of the forward pass, rounded to 32 bits, and the sums' bounds, of the terms' size
        size = np.abs(f64(dy)).sum() * np.abs(v).max() * max(1.0, float(f64(rstd).max()))
        assert abs(diff - (f64(grad) * v).sum()) <= 1e-5 * size


@pytest.mark.gpu
@pytest.mark.parametrize("n,hw,c,groups", SHAPES)
def test_mx4_form(n, hw, c, groups):
    """Codes against the 64-bit values rounded with the codes' own scale: a value is within half a step of
    its code's grid, plus its bound; a scale differs from the reference's only where the block's largest
    value lies within its bound of a power of two."""
    note(f"group norm to 4 bits {n} x {hw} x {c}, {groups} groups")
    for kind, act in (("f32", 2), ("bf16", 1), ("f16", 0)):
        x, _, w, b = case(n, hw, c, kind, n + hw + 2 * c)
        q = ifx.group_norm_mx4(x.cuda(), groups, w.cuda(), b.cuda(), 1e-5, act)
        z, _, _, tz, _, _ = forward_bounds(f64(x), groups, f64(w), f64(b), 1e-5)
        ey = lowp.act(z, act).reshape(-1, c)
        tol = (1.1 * tz + (np.abs(z) + 4) * 4 * E * np.abs(lowp.act(z, act))).reshape(-1, c)
        codes, scales = q.codes.cpu().numpy(), q.scales.cpu().numpy().astype(np.int64)
        k1, rows = (c + 127) // 128, n * hw
        assert codes.shape == (k1, rows, 64) and scales.shape == (k1, rows, 4)
        pad = ((0, 0), (0, k1 * 128 - c))
        vb = np.pad(ey, pad).reshape(rows, k1, 4, 32)
        tb = np.pad(tol, pad).reshape(rows, k1, 4, 32)
        got = np.stack((codes & 15, codes >> 4), -1).reshape(k1, rows, 4, 32).transpose(1, 0, 2, 3)
        s = scales.transpose(1, 0, 2)
        low, high = (np.abs(vb) - tb).max(-1), (np.abs(vb) + tb).max(-1)

        def scale_of(top):
            return np.where(top > 0, np.maximum(0, np.frexp(np.where(top > 0, top, 1))[1] - 1 + 125), 0)
        assert (s >= scale_of(low)).all() and (s <= scale_of(high)).all()
        unit = np.ldexp(1.0, s - 127)[..., None]
        mag = lowp.LEVELS[got & 7]
        val = mag * np.where(got & 8, -1, 1) * unit
        step = np.where(mag < 2, 0.25, np.where(mag < 4, 0.5, 1.0)) * unit  # half a step above the level
        top = (mag == 6) & (np.abs(vb) >= 6 * unit)  # saturated
        # below a level where the step changes the nearer neighbour is half as far: the wider bound covers both
        assert ((np.abs(vb - val) <= step * (1 + 1e-12) + tb) | top).all()
        assert not got.reshape(rows, -1)[:, c:].any()
        assert not s.reshape(rows, -1)[:, (c + 31) // 32:].any()


@pytest.mark.gpu
def test_no_parameters_in_place_and_other_stream():
    """weight and bias left out, y over x and dx over dy, channel slices of wider tensors, another stream."""
    n, hw, c, groups = 3, 50, 40, 8
    x, dy, _, _ = case(n, hw, c, "bf16", 1)
    one, zero = torch.ones(c), torch.zeros(c)
    wide = torch.full((n, hw, c + 7), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[..., 3:3 + c] = x.cuda()
    dwide = torch.full((n, hw, c + 9), 5.0, dtype=torch.bfloat16, device="cuda")
    dwide[..., 1:1 + c] = dy.cuda()
    xs, dys = wide[..., 3:3 + c], dwide[..., 1:1 + c]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = ifx.group_norm(xs, groups, act=ifx.ACT_SILU, stream=s)
    q = ifx.group_norm_mx4(xs, groups, act=ifx.ACT_SILU, stream=s)
    dx, dw, db = ifx.group_norm_backward(dys, xs, mean, rstd, groups, act=ifx.ACT_SILU, out=dys, stream=s.cuda_stream)
    y2, _, _ = ifx.group_norm(xs, groups, act=ifx.ACT_SILU, out=xs, stream=s)
    s.synchronize()
    check_forward(x, groups, one, zero, 1e-5, 2, y, mean, rstd, "bf16")
    check_backward(dy, x, mean.cpu(), rstd.cpu(), groups, one, zero, 2, dx, dw, db, "bf16")
    assert dx.data_ptr() == dys.data_ptr() and torch.equal(xs, y) and y2.data_ptr() == xs.data_ptr()
    for t, a in ((wide, 3), (dwide, 1)):
        assert (t[..., :a] == 5).all() and (t[..., a + c:] == 5).all()
    assert torch.equal(ifx.mx4_dequantize(q), ifx.mx4_dequantize(ifx.group_norm_mx4(x.cuda(), groups, act=ifx.ACT_SILU)))


@pytest.mark.gpu
@pytest.mark.parametrize("hw", [40, 9000])
def test_large_means_constants_and_non_finite(hw):
    """A mean far above the spread keeps its variance; a constant group gives rstd = 1 / sqrt(eps) and y = bias; a
    NaN or an infinity spoils its own sample's group alone, in codes its blocks."""
    n, c, groups = 2, 64, 2
    note(f"group norm, large means, hw = {hw}")
    x, _, w, b = case(n, hw, c, "f32", 3)
    far = (x + 3000.0).float()
    y, mean, rstd = ifx.group_norm(far.cuda(), groups, w.cuda(), b.cuda(), 1e-5, 0)
    check_forward(far, groups, w, b, 1e-5, 0, y, mean, rstd, "f32")
    flat = torch.full((n, hw, c), 7.0)
    y, mean, rstd = ifx.group_norm(flat.cuda(), groups, w.cuda(), b.cuda(), 1e-4, 0)
    assert (mean == 7).all() and np.allclose(f64(rstd), 100.0, rtol=1e-6)
    assert torch.equal(y.cpu(), b.expand(n, hw, c))
    for bad in (float("nan"), float("inf"), -float("inf")):
        z = x.clone()
        z[1, hw // 2, 3] = bad
        y, mean, rstd = ifx.group_norm(z.cuda(), groups, w.cuda(), b.cuda(), 1e-5, 2)
        check_forward(x[:1], groups, w, b, 1e-5, 2, y[:1], mean[:1], rstd[:1], "f32")
        assert torch.isnan(y[1, :, :32]).all() and torch.isfinite(y[1, :, 32:]).all()
        s = ifx.group_norm_mx4(z.cuda(), groups, w.cuda(), b.cuda(), 1e-5, 2).scales.cpu().numpy()
        assert (s[0, hw:, 0] == 255).all() and (s[0, hw:, 1] != 255).all() and (s[0, :hw] != 255).all()


@pytest.mark.gpu
def test_empty_batch_and_refusals():
    x = torch.empty(0, 5, 16, device="cuda")
    y, mean, rstd = ifx.group_norm(x, 4)
    assert y.shape == x.shape and mean.shape == (0, 4)
    assert ifx.group_norm_mx4(x, 4).codes.shape == (1, 0, 64)
    dx, dw, db = ifx.group_norm_backward(x, x, mean, rstd, 4)
    torch.cuda.synchronize()
    assert dx.shape == x.shape and not dw.any() and not db.any()
    x = torch.zeros(2, 5, 16, device="cuda")
    with pytest.raises(ifx.IfxError):
        ifx.group_norm(x, 5)
    with pytest.raises(ifx.IfxError):
        ifx.group_norm(x, 4, act=7)
    with pytest.raises(ValueError):
        ifx.group_norm(x, 4, weight=torch.ones(15, device="cuda"))
    with pytest.raises(ValueError):
        ifx.group_norm(x.transpose(1, 2), 5)
    with pytest.raises(ValueError):
        ifx.group_norm(x, 4, out=torch.empty(2, 5, 16, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ifx.group_norm_backward(x, x, torch.zeros(2, 5, device="cuda"), torch.zeros(2, 4, device="cuda"), 4)
    with pytest.raises(ValueError):
        ifx.group_norm_mx4(x, 4, out=ifx.mx4_empty(9, 16))


@pytest.mark.gpu
def test_same_from_call_to_call_and_in_a_graph():
    n, hw, c, groups = 2, 3000, 96, 12
    x, dy, w, b = (t.cuda() for t in case(n, hw, c, "bf16", 4))

    def both():
        y, mean, rstd = ifx.group_norm(x, groups, w, b, 1e-5, ifx.ACT_SILU)
        return y, mean, rstd, *ifx.group_norm_backward(dy, x, mean, rstd, groups, w, b, ifx.ACT_SILU)
    first = both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for i in range(4):
        if i > 1:
            x.mul_(1.25)
        for t in out:
            t.zero_()
        g.replay()
        expect = both()
        torch.cuda.synchronize()
        for p, q in zip(out, expect):
            assert torch.equal(p, q)
        if i < 2:
            for p, q in zip(out, first):
                assert torch.equal(p, q)


# ------------------------------------------------------------------------------------------ dispatch

def slab_of(name):
    """(gradient, threads, vectors, type, 4-bit, mode) of a slab kernel's name, None of another's."""
    m = re.match(r"gn_(grad_)?slab_kernel<(\d+), (\d+), (\d+), (?:(true|false), )?\(ifx::Mode\)(\d)>$", name)
    return m and (m[1] is not None, int(m[2]), int(m[3]), int(m[4]), m[5] == "true", int(m[6]))


def check_dispatch(n, hw, c, groups, kind, form):
    """The instance that a call launches is of its tensors' type and of the mode its groups allow, keeps no more
    registers of values than the kernels' launch bounds leave, and holds every pixel of one of the spans of whole
    groups that a sample can be cut into."""
    d = ifx.GnDesc(n, hw, c, groups, kind, 0, 1e-5, c, c, c)
    name, cg = ifx.group_norm_kernel_name(d, form), c // groups
    what = (n, hw, c, groups, kind, form, name)
    s = slab_of(name)
    if s is None:
        m = re.match(r"gn_(stats|grad_sums)_kernel<(\d+), (\d+), ", name)
        assert m and (m[1] == "grad_sums") == (form == 1) and int(m[3]) == kind, what
        assert int(m[2]) >= (c + 7) // 8, what
        return name
    grad, threads, vectors, of, mx4, mode = s
    assert of == kind and grad == (form == 1) and mx4 == (form == 2), what
    assert vectors * (8 if kind == 0 else 4) * (2 if grad else 1) <= 64, what
    fits = False
    for gs in (g for g in range(1, groups + 1) if groups % g == 0):
        cs = gs * cg
        if mx4 and cs % 32 and gs < groups:
            continue
        tcv = (cs + 7) // 8 + ((c + 127) // 128 * 16 - (c + 7) // 8 if mx4 else 0)
        m = 2 if cg % 8 == 0 else 1 if cs % 8 == 0 else 0
        fits = fits or (tcv <= threads // 4 and threads // tcv * vectors >= hw and m == mode)
    assert fits, what
    return name


# (n, hw, c, groups) at the edges of the gradient's slabs: one or a few wide groups over few pixels, spans whose last
# pixels only the widest workgroup holds
EDGES = [(8, 8, 2048, 1), (8, 1, 1536, 1), (2, 8, 2048, 1), (1, 18, 876, 1), (1, 8, 2620, 2), (1, 33, 3696, 8), (64, 42, 764, 2),
         (2, 7, 1036, 1), (40, 41, 1520, 4), (2, 169, 384, 4), (1, 169, 96, 1), (2, 225, 72, 1), (3, 9, 1100, 1), (2, 2, 2047, 1)]


def test_every_plan_has_its_kernel():
    seen = set()
    rng = random.Random(5)
    shapes = EDGES + SHAPES + [(1, hw, c, g) for hw in (1, 2, 5, 8, 9, 14, 42, 169, 340, 1024, 2100) for g in (1, 2, 4, 8, 32)
                               for c in (g, 8 * g, 12 * g, 31 * g, 96 * g, 1032, 1100, 1536, 2048, 8192) if c % g == 0 and c <= 8192]
    for _ in range(3000):
        g = rng.choice((1, 2, 4, 8, 12, 32))
        shapes.append((int(2 ** rng.uniform(0, 9)), int(2 ** rng.uniform(0, 12)), g * max(1, int(2 ** rng.uniform(0, 13)) // g), g))
    for n, hw, c, groups in shapes:
        for kind in (0, 1, 2):
            for form in (0, 1, 2):
                seen.add(check_dispatch(n, hw, c, groups, kind, form))
    # the sweep has to reach what the gradient can choose: both kinds of group in the widest workgroup, each type
    for kind in (0, 1, 2):
        assert f"gn_grad_slab_kernel<1024, 2, {kind}, (ifx::Mode)2>" in seen
        assert any(f"gn_grad_slab_kernel<1024, 2, {kind}, (ifx::Mode){m}>" in seen for m in (0, 1))


def test_kernel_name_refusals():
    d = ifx.GnDesc(1, 9, 8, 4, 1, 0, 1e-5, 8, 8, 8)
    L, buf = ifx.lib(), ctypes.create_string_buffer(256)
    assert L.ifx_group_norm_kernel_name(ctypes.byref(d), 0, buf, 256) == 0
    assert L.ifx_group_norm_kernel_name(ctypes.byref(d), 3, buf, 256) == 3 and L.ifx_group_norm_kernel_name(ctypes.byref(d), -1, buf, 256) == 3
    assert L.ifx_group_norm_kernel_name(None, 0, buf, 256) == 1 and L.ifx_group_norm_kernel_name(ctypes.byref(d), 0, None, 256) == 1
    assert L.ifx_group_norm_kernel_name(ctypes.byref(d), 0, buf, 4) == 5
    d.n = 0
    assert L.ifx_group_norm_kernel_name(ctypes.byref(d), 0, buf, 256) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("n,hw,c,groups", EDGES)
def test_backward_of_wide_groups_over_few_pixels(n, hw, c, groups):
    note(f"group norm gradient {n} x {hw} x {c}, {groups} groups")
    for kind, act in (("f32", 2), ("bf16", 2), ("f16", 0), ("bf16", 1)):
        x, dy, w, b = case(n, hw, c, kind, n + hw + c + groups)
        _, _, mean, rstd = lowp.group_norm(f64(x), groups, f64(w), f64(b), 1e-5)
        mean, rstd = torch.from_numpy(mean).float(), torch.from_numpy(rstd).float()
        dx, dw, db = ifx.group_norm_backward(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), groups, w.cuda(), b.cuda(), act)
        check_backward(dy, x, mean, rstd, groups, w, b, act, dx, dw, db, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("c,groups", [(64, 8), (40, 8), (33, 3)])
@pytest.mark.parametrize("hw", [40, 9000])
def test_constant_groups_of_large_values(hw, c, groups):
    """Every pixel of a group the same large value, in each type: the mean is that value (p 2^q of few bits, whose
    sums are exact as long as their count times p is below 2^24), the variance 0, and y = act(bias), however large
    rstd and the mean are; its codes are those of act(bias)."""
    n = 2
    rng = np.random.default_rng(4)
    w = torch.from_numpy(1 + 0.5 * rng.standard_normal(c)).float()
    b = torch.from_numpy(0.5 * rng.standard_normal(c)).float()
    for kind in ("f32", "bf16", "f16"):
        for value in (7.0, 1000.0, 57344.0, -57344.0):
            assert hw * c // groups * 125 < 2 ** 24
            note(f"group norm, constant {value} {kind}, {n} x {hw} x {c}, {groups} groups")
            x = torch.full((n, hw, c), value, dtype=TYPES[kind])
            for act in (0, 1, 2):
                y, mean, rstd = ifx.group_norm(x.cuda(), groups, w.cuda(), b.cuda(), 1e-5, act)
                assert (mean == value).all() and np.allclose(f64(rstd), 1e-5 ** -0.5, rtol=1e-6)
                exact = np.broadcast_to(lowp.act(f64(b), act), (n, hw, c)).copy()
                tol = (np.abs(f64(b)) + 4) * 4 * E * np.abs(exact) if act == 2 else 0 * exact
                assert excess(f64(y), exact, tol, kind) == 0
                if act < 2:
                    codes, scales = lowp.mx4_quantize(exact[0, :1])
                    q = ifx.group_norm_mx4(x.cuda(), groups, w.cuda(), b.cuda(), 1e-5, act)
                    assert (q.codes.cpu().numpy() == codes).all() and (q.scales.cpu().numpy() == scales).all()


@pytest.mark.gpu
@pytest.mark.parametrize("c,groups", [(64, 8), (40, 8), (33, 3)])
def test_nearly_constant_groups_of_large_values(c, groups):
    """Two pixels of each group off its large value by the last bit of float16, one up and one down: the mean is the
    value, exactly, and the bound has no part that grows with it."""
    n, hw, value = 2, 40, 1024.0
    cg = c // groups
    rng = np.random.default_rng(6)
    w = torch.from_numpy(1 + 0.5 * rng.standard_normal(c)).float()
    b = torch.from_numpy(0.5 * rng.standard_normal(c)).float()
    x = torch.full((n, hw, c), value)
    x[:, 3, ::cg] += 1
    x[:, 29, cg - 1::cg] -= 1
    z, xhat, mean, rstd = lowp.group_norm(f64(x), groups, f64(w), f64(b), 1e-5)
    # (mean exact: forward_bounds with d(mean) = 0 and x - mean, not x, times rstd w)
    tol = np.abs(f64(w) * xhat) * 40 * E + 4 * E * (np.abs(f64(w) * xhat) + np.abs(f64(b)))
    for kind in ("f32", "f16"):
        note(f"group norm, nearly constant {kind}, {n} x {hw} x {c}, {groups} groups")
        y, m, r = ifx.group_norm(x.to(TYPES[kind]).cuda(), groups, w.cuda(), b.cuda(), 1e-5, 0)
        assert (m == value).all() and worst(f64(r), rstd, 40 * E * rstd) <= 1
        assert excess(f64(y), z, tol, kind) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("c,groups", [(64, 8), (33, 3)])
@pytest.mark.parametrize("hw", [40, 9000])
def test_means_whose_square_overflows(hw, c, groups):
    """A mean of 2^67, whose square is past float32: the variance is that of the differences, whose squares are not."""
    n = 2
    x, _, w, b = case(n, hw, c, "f32", 12)
    note(f"group norm, mean 2^67, {n} x {hw} x {c}, {groups} groups")
    for kind in ("f32", "bf16"):
        flat = torch.full((n, hw, c), 2.0 ** 67, dtype=TYPES[kind])
        y, mean, rstd = ifx.group_norm(flat.cuda(), groups, w.cuda(), b.cuda(), 1e-5, 0)
        assert (mean == 2.0 ** 67).all() and np.allclose(f64(rstd), 1e-5 ** -0.5, rtol=1e-6)
        assert torch.equal(y.cpu(), b.to(TYPES[kind]).expand(n, hw, c))
    far = (x.double() * 2.0 ** 54 + 2.0 ** 67).float()
    y, mean, rstd = ifx.group_norm(far.cuda(), groups, w.cuda(), b.cuda(), 1e-5, 1)
    check_forward(far, groups, w, b, 1e-5, 1, y, mean, rstd, "f32")


def test_workspace_of_the_4_bit_form_needs_no_ld_y():
    """The 4-bit form has no y: a descriptor without its pitch is valid for it, and so is the query's answer."""
    L, fake = ifx.lib(), ctypes.c_void_p(0x100000)
    for n, hw, c, groups in ((3, 100003, 64, 8), (1, 16384, 512, 32), (1, 5000, 33, 3)):
        full, none = (ifx.GnDesc(n, hw, c, groups, 1, 0, 1e-5, c, ld_y, 0) for ld_y in (c, 0))
        need = L.ifx_group_norm_workspace_bytes(ctypes.byref(none), 0)
        assert 0 < need <= L.ifx_group_norm_workspace_bytes(ctypes.byref(full), 0)
        # far enough to ask for the codes: not IFX_E_WORKSPACE
        assert L.ifx_group_norm_mx4(ctypes.byref(none), fake, None, None, None, fake, None, None, fake, need, None) == 1
        assert L.ifx_group_norm(ctypes.byref(none), fake, None, None, fake, None, None, fake, 1 << 40, None) == 2
    assert L.ifx_group_norm_workspace_bytes(ctypes.byref(ifx.GnDesc(1, 9, 8, 4, 1, 0, 1e-5, 7, 0, 0)), 0) == 0


HOST_ONLY = r"""
#include <dlfcn.h>
#include <stdio.h>
#include "ifx.h"
/* takes the runtime's place: a device of 32 compute units, and a count of who asks */
static int asked;
int hipGetDevice(int *dev) { ++asked; *dev = 0; return 0; }
int hipDeviceGetAttribute(int *v, int attr, int dev) { ++asked; *v = 32; return 0; }
int hipGetDeviceCount(int *n) { ++asked; *n = 1; return 0; }
int main(int argc, char **argv)
{
    void *l = dlopen(argv[1], RTLD_NOW);
    if (!l) { puts(dlerror()); return 1; }
    size_t (*bytes)(const ifx_gn_desc *, int32_t) = (size_t (*)(const ifx_gn_desc *, int32_t))dlsym(l, "ifx_group_norm_workspace_bytes");
    ifx_status (*norm)(const ifx_gn_desc *, const void *, const float *, const float *, void *, float *, float *, void *, size_t, void *) =
        (ifx_status (*)(const ifx_gn_desc *, const void *, const float *, const float *, void *, float *, float *, void *, size_t, void *))dlsym(l, "ifx_group_norm");
    ifx_gn_desc d = {0};
    int n, hw, c, groups;
    asked = 0;
    while (scanf("%d %d %d %d", &n, &hw, &c, &groups) == 4) {
        d.n = n, d.hw = hw, d.c = c, d.groups = groups, d.type = IFX_BF16, d.ld_x = d.ld_y = d.ld_dy = c;
        printf("%zu %zu %d\n", bytes(&d, 0), bytes(&d, 1), (int)norm(&d, &d, 0, 0, 0, 0, 0, 0, 0, 0));
    }
    printf("asked %d\n", asked);
    return 0;
}
"""


def test_validation_touches_no_device(tmp_path):
    """The workspace query and the checks of a call ask the runtime nothing, so a workspace sized under one device
    serves any other."""
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "host.c", tmp_path / "host"
    src.write_text(HOST_ONLY)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-rdynamic", "-I", os.path.join(root, "include"), str(src), "-o", str(exe), "-ldl"], check=True)
    ifx.lib()
    shapes = SHAPES + [(1, 3136, 256, 32), (32, 3136, 256, 32), (2, 3136, 256, 32), (64, 784, 512, 32)]
    r = subprocess.run([str(exe), ifx.LIB_PATH], input="\n".join(" ".join(map(str, s)) for s in shapes), capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    *lines, asked = r.stdout.split("\n")[:-1]
    assert asked == "asked 0"
    for (n, hw, c, groups), line in zip(shapes, lines, strict=True):
        d = ifx.GnDesc(n, hw, c, groups, 1, 0, 0.0, c, c, c)
        forward, backward, status = map(int, line.split())
        assert [forward, backward] == [ifx.lib().ifx_group_norm_workspace_bytes(ctypes.byref(d), i) for i in (0, 1)], (n, hw, c, groups)
        assert status == 5 or status == 1  # no workspace where some is needed, or no y
