"""Microscaled 4-bit tensors: the 64-bit reference's own pins and the entry points' refusals (CPU), and the
kernels against the reference (GPU).

Codes, scales and the values back are compared bit for bit.  A product's bound: with S the sum of the
magnitudes of its terms (bias and residual among them), every one of its roundings, K1 = ceil(k / 128)
matrix instructions (whose own error was measured at most 2^-23 S), the joins of at most 16 partial sums and two
additions, is off by at most 2^-23 S, so |z - exact| <= (K1 + 18) 2^-23 S; SiLU stretches that by at most
1.1 and adds (|z| + 4) 2^-22 |y| for its exponential and division; then one rounding to the type.
"""
import ctypes
import sys

import numpy as np
import pytest
import torch

import convolution_int8_implicit_amd as ifx
from oracle import lowp

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


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


def tensor_of(q, k, device="cuda"):
    return ifx.Mx4(torch.from_numpy(q[0].copy()).to(device), torch.from_numpy(q[1].copy()).to(device), k)


# ------------------------------------------------------------------------------------------ CPU

def test_reference_rounding_pins():
    """Halves go to the even code, magnitudes past 6 saturate, the scale is the largest magnitude's."""
    x = np.zeros((1, 32))
    x[0, :10] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26, 7.9]
    codes, scales = lowp.mx4_quantize(x)
    assert codes.shape == (1, 1, 64) and scales.shape == (1, 1, 4)
    assert list(scales[0, 0]) == [127, 0, 0, 0]
    v = lowp.mx4_values(codes, scales, 32)[0]
    assert list(v[:10]) == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.5, 6.0]
    assert codes[0, 0, 0] == 7 and codes[0, 0, 4] == (8 + 1) + 16 * 7
    # powers of two: 2^e has scale e - 2 and code 6 (4.0)
    for e in (-126, -3, 0, 5, 127):
        c, s = lowp.mx4_quantize(np.array([[2.0 ** e]]))
        assert s[0, 0, 0] == max(0, e - 2 + 127) and lowp.mx4_values(c, s, 1)[0, 0] == 2.0 ** e
    c, s = lowp.mx4_quantize(np.array([[1.0, np.inf], [np.nan, 0.0]]))
    assert list(s[0, :, 0]) == [255, 255] and not c.any()
    c, s = lowp.mx4_quantize(np.array([[-0.0, 0.0]]))
    assert s[0, 0, 0] == 0 and c[0, 0, 0] == 8


def test_reference_values_are_fixed_points():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 200)) * 10.0 ** rng.integers(-8, 8, (5, 200))
    q = lowp.mx4_quantize(x)
    v = lowp.mx4_values(*q, 200)
    again = lowp.mx4_quantize(v)
    assert np.array_equal(lowp.mx4_values(*again, 200), v)
    top = np.abs(np.pad(x, ((0, 0), (0, 24))).reshape(5, 7, 32)).max(-1, keepdims=True)
    assert (np.abs(np.pad(v - x, ((0, 0), (0, 24))).reshape(5, 7, 32)) <= top / 4).all()


def test_sizes_and_refusals_need_no_device():
    L = ifx.lib()
    fake, odd, half = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001), ctypes.c_void_p(0x100002)
    assert L.ifx_mx4_code_bytes(5, 129) == 2 * 5 * 64 and L.ifx_mx4_scale_bytes(5, 129) == 2 * 5 * 4
    assert L.ifx_mx4_code_bytes(-1, 5) == 0 and L.ifx_mx4_scale_bytes(1, 0) == 0
    for fn, args in ((L.ifx_mx4_quantize, lambda x, t, ld, r, k, c, s: (x, t, ld, r, k, c, s, None)),
                     (L.ifx_mx4_dequantize, lambda x, t, ld, r, k, c, s: (c, s, r, k, x, t, ld, None))):
        assert fn(*args(None, 0, 4, 1, 4, fake, fake)) == 1
        assert fn(*args(fake, 0, 4, 1, 4, None, fake)) == 1
        assert fn(*args(fake, 0, 4, 1, 4, fake, None)) == 1
        assert fn(*args(fake, 3, 4, 1, 4, fake, fake)) == 3
        assert fn(*args(fake, 0, 3, 1, 4, fake, fake)) == 2
        assert fn(*args(fake, 0, 4, -1, 4, fake, fake)) == 2
        assert fn(*args(fake, 0, 4, 1, 0, fake, fake)) == 2
        assert fn(*args(fake, 0, 1 << 61, 4, 4, fake, fake)) == 2
        assert fn(*args(fake, 0, 1 << 30, (1 << 31) - 1, 1 << 30, fake, fake)) == 2
        assert fn(*args(half, 0, 4, 1, 4, fake, fake)) == 4
        assert fn(*args(odd, 1, 4, 1, 4, fake, fake)) == 4
        assert fn(*args(fake, 1, 4, 1, 4, ctypes.c_void_p(0x100008), fake)) == 4
        assert fn(*args(fake, 1, 4, 1, 4, fake, half)) == 4
        assert fn(*args(None, 1, 4, 0, 4, None, None)) == 0

    def mm(m=2, n=3, k=4, t=1, act=0, ld_y=3, ld_res=3, a=fake, asc=fake, w=fake, wsc=fake, bias=fake, res=fake, y=fake):
        return L.ifx_mx4_matmul(ctypes.byref(ifx.Mx4Desc(m, n, k, t, act, ld_y, ld_res)), a, asc, w, wsc, bias, res, y,
                                None)
    assert L.ifx_mx4_matmul(None, fake, fake, fake, fake, None, None, fake, None) == 1
    for name in ("a", "asc", "w", "wsc", "y"):
        assert mm(**{name: None}) == 1, name
    assert mm(t=5) == 3 and mm(act=3) == 3 and mm(act=-1) == 3
    assert mm(m=-1) == 2 and mm(n=-1) == 2 and mm(k=0) == 2 and mm(ld_y=2) == 2 and mm(ld_res=2) == 2
    assert mm(y=odd) == 4 and mm(res=odd) == 4 and mm(bias=half) == 4 and mm(a=half) == 4 and mm(wsc=half) == 4
    assert mm(m=0, a=None, y=None) == 0 and mm(n=0, ld_y=0, ld_res=0, w=None) == 0


def test_a_grid_past_the_launch_limit_is_refused():
    """2^32 - 1 work-items: 64 x 64 tiles of 256 threads, with room for the deal over eight XCDs."""
    L = ifx.lib()
    fake = ctypes.c_void_p(0x100000)

    def mm(m, n):
        d = ifx.Mx4Desc(m, n, 64, 1, 0, n, n)
        return L.ifx_mx4_matmul(ctypes.byref(d), fake, fake, fake, fake, None, None, None, None)
    assert mm(1 << 18, 1 << 17) == 1          # 2^23 tiles: goes on to the NULL y
    assert mm(1 << 18, 1 << 18) == 2 and mm(1 << 27, 1 << 10) == 2


def test_binding_refusals_need_no_device():
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        ifx.mx4_quantize(x)  # not on a GPU
    with pytest.raises(ValueError):
        ifx._pitch(torch.zeros(4, 32).t())
    with pytest.raises(ValueError):
        ifx._pitch(torch.zeros(1, 32).expand(4, 32))
    with pytest.raises(ValueError):
        ifx._pitch(torch.zeros(4, 6, 32)[:, :5])
    assert ifx._pitch(torch.zeros(4, 6, 32)[..., 3:20]) == (24, 17, 32)
    assert ifx._pitch(torch.zeros(4, 1, 32)[:, :, 1:]) == (4, 31, 32)
    assert ifx._pitch(torch.zeros(0, 32)) == (0, 32, 32)
    with pytest.raises(TypeError):
        ifx._type(torch.int8)
    with pytest.raises(ValueError):
        ifx._mx4_check(ifx.Mx4(torch.zeros(1, 4, 64, dtype=torch.uint8), torch.zeros(1, 3, 4, dtype=torch.uint8), 32), "a")
    with pytest.raises(ValueError):
        ifx._mx4_check(ifx.Mx4(torch.zeros(1, 4, 64, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8), 129), "a")


# ------------------------------------------------------------------------------------------ GPU

def block_values(rows, k, kind, seed):
    """Values of every magnitude that the type holds, among them zeros, exact halves between levels,
    subnormals, the type's extremes, infinities and NaN (one block each)."""
    rng = np.random.default_rng(seed)
    low, high = {"f32": (-148, 126), "bf16": (-132, 126), "f16": (-23, 13)}[kind]
    x = rng.standard_normal((rows, k)) * 2.0 ** rng.integers(low + 3, high, (rows, 1))
    pick = rng.random((rows, k))
    unit = 2.0 ** rng.integers(low + 3, high - 3, (rows, 1))
    x = np.where(pick < 0.3, unit * rng.choice([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.5],
                                               (rows, k)) * rng.choice([-1, 1], (rows, k)), x)
    x = np.where(pick > 0.97, 0.0, x)
    t = torch.from_numpy(x).to(TYPES[kind])
    if rows > 4:
        t[1, k // 2] = float("nan")
        t[2, 0] = float("inf")
        t[3, k - 1] = -float("inf")
        t[4] = 0
        t[4, 0] = -0.0
        t[rows - 1, 0] = torch.finfo(TYPES[kind]).max
        t[rows - 1, k - 1] = torch.finfo(TYPES[kind]).min
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 2048), (7, 31), (5, 33), (17, 128), (33, 130), (16, 515), (50, 997)])
def test_quantize(rows, k, kind):
    note(f"quantize {rows} x {k} {kind}")
    x = block_values(rows, k, kind, 7 * rows + k)
    codes, scales = lowp.mx4_quantize(f64(x))
    q = ifx.mx4_quantize(x.cuda())
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    v = lowp.mx4_values(codes, scales, k)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        with np.errstate(over="ignore", invalid="ignore"):
            # float64 to float16 in one rounding; the others hold the values exactly
            expect = v.astype(np.float16).astype(np.float64) if dtype == torch.float16 else v
        got = ifx.mx4_dequantize(q, dtype)
        assert got.shape == (rows, k) and got.dtype == dtype
        assert np.array_equal(f64(got), expect, equal_nan=True)


@pytest.mark.gpu
def test_quantize_every_float16():
    """Every finite float16, a block each of it and of half its magnitude."""
    bits = np.arange(65536, dtype=np.uint16)
    v = bits.view(np.float16)
    v = v[np.isfinite(v)]
    x = np.zeros((v.size, 32), dtype=np.float16)
    x[:, 0], x[:, 5] = v, v / np.float16(2)
    x[:, 9] = v * np.float16(0.3125)
    q = ifx.mx4_quantize(torch.from_numpy(x).cuda())
    top = np.abs(x.astype(np.float64)).max(1)
    s = np.where(top > 0, np.frexp(np.where(top > 0, top, 1))[1] - 1 + 125, 0)
    assert np.array_equal(q.scales.cpu().numpy()[0, :, 0], s)
    unit = np.abs(np.ldexp(x.astype(np.float64), (127 - s)[:, None]))
    code = sum((unit > t) | ((unit == t) & even) for t, even in ((.25, False), (.75, True), (1.25, False), (1.75, True),
                                                                 (2.5, False), (3.5, True), (5.0, False)))
    code = code + 8 * np.signbit(x)
    got = q.codes.cpu().numpy()[0]
    got = np.stack((got & 15, got >> 4), -1).reshape(v.size, 128)
    assert np.array_equal(got[:, :32], code) and not got[:, 32:].any()


@pytest.mark.gpu
def test_quantize_strides_streams_and_out():
    """A slice of a wider tensor at an odd offset, more axes than two, another stream, given outputs."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(3, 5, 7, 301, device="cuda", generator=gen).to(torch.bfloat16)
    x = wide[..., 3:300]
    codes, scales = lowp.mx4_quantize(f64(x).reshape(-1, 297))
    out = ifx.mx4_empty(105, 297)
    out.codes.fill_(0xAA)
    out.scales.fill_(0xAA)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = ifx.mx4_quantize(x, out=out, stream=s)
    dst = torch.full((105, 400), 7.0, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    ifx.mx4_dequantize(q, out=dst[:, 1:298], stream=s.cuda_stream)
    s.synchronize()
    assert q.codes is out.codes
    assert np.array_equal(out.codes.cpu().numpy(), codes) and np.array_equal(out.scales.cpu().numpy(), scales)
    assert np.array_equal(f64(dst[:, 1:298]), lowp.mx4_values(codes, scales, 297))
    assert (dst[:, 0] == 7).all() and (dst[:, 298:] == 7).all()


@pytest.mark.gpu
def test_quantize_empty_and_refusals():
    q = ifx.mx4_quantize(torch.empty(0, 64, device="cuda"))
    assert q.codes.shape == (1, 0, 64) and ifx.mx4_dequantize(q).shape == (0, 64)
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError):
        ifx.mx4_quantize(x.t())
    with pytest.raises(ValueError):
        ifx.mx4_quantize(x, out=ifx.mx4_empty(5, 64))
    with pytest.raises(TypeError):
        ifx.mx4_quantize(x.double())
    with pytest.raises(ifx.IfxError):
        ifx.mx4_quantize(torch.empty(4, 0, device="cuda"), out=None)


def product_case(m, n, k, seed, zero_row=True):
    rng = np.random.default_rng(seed)
    k1 = (k + 127) // 128

    def one(rows):
        x = rng.standard_normal((rows, k)) * 2.0 ** rng.integers(-6, 6, (rows, 1))
        if rows > 2 and zero_row:
            x[1] = 0
        codes = rng.integers(0, 256, (k1, rows, 64), dtype=np.uint8)
        scales = rng.integers(118, 134, (k1, rows, 4), dtype=np.uint8)
        # the padding of the last columns: zero codes
        col = np.arange(k1 * 128).reshape(k1, 1, 64, 2)
        codes = np.where(col[..., 0] < k, codes & 15, 0) | np.where(col[..., 1] < k, codes & 240, 0)
        scales[(np.arange(k1 * 4).reshape(k1, 1, 4) * 32 >= k).repeat(rows, 1)] = 0
        if rows > 2 and zero_row:
            codes[:, 1] = 0
        return codes.astype(np.uint8), scales
    return one(m), one(n), rng.standard_normal(n).astype(np.float32) * 30, rng.standard_normal((m, n)) * 30


def check_product(y, m, n, k, a, w, bias, res, act, kind):
    exact, z, s = lowp.mx4_matmul(a, w, k, bias, res, act)
    tol = ((k + 127) // 128 + 18) * 2.0 ** -23 * s
    if act == ifx.ACT_SILU:
        tol = 1.1 * tol + (np.abs(z) + 4) * 2.0 ** -22 * np.abs(exact)
    got = f64(y)
    assert got.shape == (m, n)
    assert (np.isnan(got) == np.isnan(exact)).all()
    assert excess(got, exact, tol, kind) == 0


SHAPES = [(1, 1, 1), (1, 40, 2048), (2, 17, 33), (5, 1000, 130), (16, 16, 128), (17, 31, 129), (33, 65, 640),
          (64, 64, 256), (65, 130, 96), (100, 300, 1000), (130, 257, 385), (257, 129, 512), (300, 520, 64),
          # enough tiles for the larger ones, edges inside a tile, one to seven steps of the ring
          (2050, 2049, 300), (2111, 1930, 900), (4097, 4100, 130), (4200, 3970, 600)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul(m, n, k):
    note(f"product {m} x {n} x {k}")
    a, w, bias, res = product_case(m, n, k, m + 3 * n + 7 * k)
    A, W = tensor_of(a, k), tensor_of(w, k)
    for i, (kind, act) in enumerate((("f32", 0), ("bf16", 1), ("f16", 2))):
        b = bias if i != 1 or m % 2 else None
        scale = 0.01 if kind == "f16" else 1.0  # keeps float16 results finite
        wq = (w[0], w[1] - 7 * (w[1] > 0).astype(np.uint8)) if kind == "f16" else w
        r = torch.from_numpy(res * scale).to(TYPES[kind]) if (i + n) % 2 else None
        y = ifx.mx4_matmul(A, tensor_of(wq, k) if kind == "f16" else W, None if b is None else torch.from_numpy(b).cuda(),
                           None if r is None else r.cuda(), act, TYPES[kind])
        check_product(y, m, n, k, a, wq, b, None if r is None else f64(r), act, kind)


@pytest.mark.gpu
def test_matmul_long_sums():
    """The tile for long sums: every step of the ring many times over, ragged edges; rows and columns sampled."""
    m, n, k = 4100, 4090, 4200
    note(f"product {m} x {n} x {k}")
    a, w, bias, res = product_case(m, n, k, 77)
    rows = np.unique(np.r_[0:3, 255:258, 2047:2050, m - 5:m, np.random.default_rng(2).integers(0, m, 40)])
    some = tuple(np.ascontiguousarray(t[:, rows]) for t in a)
    for kind, act in (("f32", 0), ("bf16", 1)):
        r = torch.from_numpy(res).to(TYPES[kind])
        y = ifx.mx4_matmul(tensor_of(a, k), tensor_of(w, k), torch.from_numpy(bias).cuda(), r.cuda(), act, TYPES[kind])
        check_product(y[torch.from_numpy(rows).cuda()], len(rows), n, k, some, w, bias, f64(r)[rows], act, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 40, 300])
def test_matmul_nan_blocks_and_extreme_scales(m):
    """A NaN scale spoils its row or column alone; scales of 0 and 252 multiply exactly."""
    n, k = 70, 300
    note(f"product with NaN blocks, m = {m}")
    a, w, _, _ = product_case(m, n, k, 11 + m)
    w[1][1, 5, 2] = 255
    w[1][2, n - 1, 0] = 255
    if m > 3:
        a[1][0, 3, 1] = 255
    y = f64(ifx.mx4_matmul(tensor_of(a, k), tensor_of(w, k), dtype=torch.float32))
    nan = np.zeros((m, n), dtype=bool)
    nan[:, [5, n - 1]] = True
    if m > 3:
        nan[3] = True
    assert (np.isnan(y) == nan).all()
    check_product(torch.from_numpy(y), m, n, k, a, w, None, None, 0, "f32")
    a[1][a[1] > 0] = 252
    w[1][w[1] > 0] = 3
    check_product(ifx.mx4_matmul(tensor_of(a, k), tensor_of(w, k), dtype=torch.float32), m, n, k, a, w, None, None, 0,
                  "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,off", [(3, 50, 1), (200, 130, 3), (300, 256, 8)])
def test_matmul_pitches_in_place_and_stream(m, n, off):
    """The output a slice of a wider tensor at an odd offset, the residual that same memory, another stream:
    nothing outside the slice is written."""
    k = 260
    a, w, bias, res = product_case(m, n, k, 5)
    s = torch.cuda.Stream()
    for kind in ("bf16", "f32"):
        note(f"product into a slice, {m} x {n} {kind}")
        wide = torch.full((m, n + 2 * off + 5), 3.0, dtype=TYPES[kind], device="cuda")
        y = wide[:, off:off + n]
        y.copy_(torch.from_numpy(res))
        r = f64(y)
        A, W, B = tensor_of(a, k), tensor_of(w, k), torch.from_numpy(bias).cuda()
        s.wait_stream(torch.cuda.current_stream())
        got = ifx.mx4_matmul(A, W, B, y, ifx.ACT_RELU, out=y, stream=s)
        s.synchronize()
        assert got.data_ptr() == y.data_ptr()
        check_product(y, m, n, k, a, w, bias, r, 1, kind)
        assert (wide[:, :off] == 3).all() and (wide[:, off + n:] == 3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("pitch", [128, 136])
def test_results_larger_than_the_caches(pitch):
    """Results of 18 MB and more in rows that fill 128-byte lines and rows that share them, their last columns and
    last rows inside a tile."""
    m, n, k = 70001, 125, 64
    a, w, bias, res = product_case(m, n, k, 11)
    A, W = tensor_of(a, k), tensor_of(w, k)
    for kind, with_res in (("bf16", False), ("f16", True), ("f32", True)):
        note(f"product {m} x {n} x {k} {kind}, rows of {pitch}")
        wq = (w[0], w[1] - 7 * (w[1] > 0).astype(np.uint8))  # keeps float16 results finite
        r = torch.from_numpy(res * 0.01).to(TYPES[kind]) if with_res else None
        wide = torch.full((m, pitch), 3.0, dtype=TYPES[kind], device="cuda")
        ifx.mx4_matmul(A, tensor_of(wq, k), torch.from_numpy(bias).cuda(), None if r is None else r.cuda(),
                       ifx.ACT_RELU, out=wide[:, :n])
        check_product(wide[:, :n], m, n, k, a, wq, bias, None if r is None else f64(r), ifx.ACT_RELU, kind)
        assert bool((wide[:, n:] == 3).all())
    codes, scales = product_case(m, 2, 117, 12)[0]
    v = lowp.mx4_values(codes, scales, 117)
    for kind in ("bf16", "f16", "f32"):
        note(f"values {m} x 117 {kind}, rows of {pitch}")
        wide = torch.full((m, pitch), 3.0, dtype=TYPES[kind], device="cuda")
        ifx.mx4_dequantize(tensor_of((codes, scales), 117), out=wide[:, :117])
        assert np.array_equal(f64(wide[:, :117]), v.astype(np.float16).astype(np.float64) if kind == "f16" else v)
        assert bool((wide[:, 117:] == 3).all())


@pytest.mark.gpu
def test_matmul_same_from_call_to_call_and_in_a_graph():
    m, n, k = 130, 200, 1024
    a, w, bias, _ = product_case(m, n, k, 9)
    A, W, B = tensor_of(a, k), tensor_of(w, k), torch.from_numpy(bias).cuda()
    first = ifx.mx4_matmul(A, W, B)
    out = torch.empty_like(first)
    x = torch.randn(m, k, device="cuda")
    q = ifx.mx4_empty(m, k)
    ifx.mx4_quantize(x, out=q)
    other = ifx.mx4_matmul(q, W, B)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ifx.mx4_quantize(x, out=q)
        ifx.mx4_matmul(q, W, B, out=out)
    for i in range(4):
        q.codes.zero_()
        out.zero_()
        x.add_(0.0 if i < 2 else 1.0)
        g.replay()
        expect = ifx.mx4_matmul(ifx.mx4_quantize(x), W, B)
        torch.cuda.synchronize()
        assert torch.equal(out, expect)
        if i < 2:
            assert torch.equal(out, other)
        assert torch.equal(ifx.mx4_matmul(A, W, B), first)


@pytest.mark.gpu
def test_matmul_empty_and_refusals():
    W = ifx.mx4_quantize(torch.ones(6, 64, device="cuda"))
    none = ifx.mx4_quantize(torch.empty(0, 64, device="cuda"))
    assert ifx.mx4_matmul(none, W).shape == (0, 6) and ifx.mx4_matmul(W, none).shape == (6, 0)
    with pytest.raises(ValueError):
        ifx.mx4_matmul(W, ifx.mx4_quantize(torch.ones(6, 65, device="cuda")))
    with pytest.raises(ValueError):
        ifx.mx4_matmul(W, W, bias=torch.ones(5, device="cuda"))
    with pytest.raises(ValueError):
        ifx.mx4_matmul(W, W, residual=torch.ones(6, 6, device="cuda"))
    with pytest.raises(ValueError):
        ifx.mx4_matmul(W, W, residual=torch.ones(6, 6, device="cuda", dtype=torch.bfloat16).t())
    with pytest.raises(ifx.IfxError):
        ifx.mx4_matmul(W, W, act=9)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^32 bytes and 2^31 elements, and codes past 2^32 bytes."""
    rows, k = (1 << 21) + 5, 1100
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(37, k, device="cuda", generator=gen)
    x[-37:] = tail
    q = ifx.mx4_quantize(x)
    codes, scales = lowp.mx4_quantize(f64(x[-37:]))
    assert np.array_equal(q.codes[:, -37:].cpu().numpy(), codes) and np.array_equal(q.scales[:, -37:].cpu().numpy(), scales)
    assert not q.codes[:, :-37].any()
    v = ifx.mx4_dequantize(q)
    assert np.array_equal(f64(v[-37:]), lowp.mx4_values(codes, scales, k)) and not v[:-37].any()
    del x, v
    m, k = (1 << 20) + 3, 8192 + 128
    a = ifx.Mx4(torch.zeros(k // 128, m, 64, dtype=torch.uint8, device="cuda"),
                torch.zeros(k // 128, m, 4, dtype=torch.uint8, device="cuda"), k)
    assert a.codes.numel() > 1 << 32
    t = ifx.mx4_quantize(torch.randn(40, k, device="cuda", generator=gen))
    a.codes[:, -40:], a.scales[:, -40:] = t.codes, t.scales
    w = ifx.mx4_quantize(torch.randn(24, k, device="cuda", generator=gen))
    y = ifx.mx4_matmul(a, w)
    few = (t.codes.cpu().numpy(), t.scales.cpu().numpy())
    check_product(y[-40:], 40, 24, k, few, (w.codes.cpu().numpy(), w.scales.cpu().numpy()), None, None, 0, "bf16")
    assert not y[:-40].any()


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """The C entry points take 32-bit sizes: a larger tensor is refused by the binding, not taken modulo 2^32.  The
    tensors are on no device and have no memory, so a call that went on would be refused for its NULL pointers."""
    monkeypatch.setattr(ifx, "_on_device", lambda *ts: 0)
    monkeypatch.setattr(ifx, "_raw_stream", lambda stream, index: 0)

    def meta(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="meta")

    def mx4(rows, k):
        k1 = (k + 127) // 128
        return ifx.Mx4(meta(k1, rows, 64, dtype=torch.uint8), meta(k1, rows, 4, dtype=torch.uint8), k)
    big, fit = (1 << 32) + 5, 5
    calls = [lambda b: ifx.mx4_quantize(meta(b, 3)), lambda b: ifx.mx4_quantize(meta(3, b)),
             lambda b: ifx.mx4_quantize(meta(b, 3), out=mx4(b, 3)),
             lambda b: ifx.mx4_dequantize(mx4(b, 3)), lambda b: ifx.mx4_dequantize(mx4(3, b)),
             lambda b: ifx.mx4_matmul(mx4(b, 3), mx4(4, 3)), lambda b: ifx.mx4_matmul(mx4(4, 3), mx4(b, 3)),
             lambda b: ifx.mx4_matmul(mx4(4, b), mx4(4, b)), lambda b: ifx.mx4_matmul(mx4(4, 3), mx4(4, 3), act=b - fit),
             lambda b: ifx.group_norm(meta(b, 2, 8), 4), lambda b: ifx.group_norm(meta(2, b, 8), 4),
             lambda b: ifx.group_norm(meta(2, 3, b - 1), 4), lambda b: ifx.group_norm(meta(2, 3, 8), b - 1),
             lambda b: ifx.group_norm(meta(2, 3, 8), 4, act=b - fit),
             lambda b: ifx.group_norm_mx4(meta(b, 2, 8), 4), lambda b: ifx.group_norm_mx4(meta(2, b, 8), 4),
             lambda b: ifx.group_norm_backward(meta(b, 2, 8), meta(b, 2, 8), meta(b, 4), meta(b, 4), 4),
             lambda b: ifx.group_norm_backward(meta(2, b, 8), meta(2, b, 8), meta(2, 4), meta(2, 4), 4)]
    for i, call in enumerate(calls):
        with pytest.raises(ifx.IfxError, match="NULL"):
            call(fit)
        with pytest.raises(ValueError, match="32 bits"):
            call(big)
            pytest.fail(f"call {i}")


@pytest.mark.gpu
def test_longest_rows():
    """One row of 2^31 - 1 columns, the most that an int32 counts: the last panels, whose end and padding lie past
    where a column number plus a few passes 31 bits, and nothing in the panels before them."""
    k = (1 << 31) - 1
    k1 = (k - 1) // 128 + 1
    first = (k1 - 4) * 128
    note(f"one row of {k} columns")
    x = torch.zeros(1, k, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x[:, first:] = torch.randn(1, k - first, device="cuda", generator=gen)
    codes, scales = lowp.mx4_quantize(f64(x[:, first:]))
    note("rounding")
    q = ifx.mx4_quantize(x)
    assert q.codes.shape == (k1, 1, 64)
    assert np.array_equal(q.codes[-4:].cpu().numpy(), codes) and np.array_equal(q.scales[-4:].cpu().numpy(), scales)
    assert not q.codes[:-4].any() and not q.scales[:-4].any()
    del x
    note("values")
    v = ifx.mx4_dequantize(q)
    assert np.array_equal(f64(v[:, first:]), lowp.mx4_values(codes, scales, k - first)) and not v[:, :first].any()
    del v
    note("product")
    exact, _, s = lowp.mx4_matmul((codes, scales), (codes, scales), k - first)
    # the other panels add zeros: no rounding of theirs
    assert excess(f64(ifx.mx4_matmul(q, q, dtype=torch.float32)), exact, (4 + 18) * 2.0 ** -23 * s, "f32") == 0
