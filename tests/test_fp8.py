"""8-bit floating point tensors with a power of two per block of 128: the 64-bit reference's own pins and the entry
points' refusals (CPU), and the kernels against the reference (GPU).

Codes, scales and the values back are compared bit for bit.  A product's bound, with S the sum of the magnitudes of its
terms (bias and residual among them) and K1 = ceil(k / 128): a matrix instruction (2 a panel on 8-bit operands, 8 on
bfloat16 ones), a join of two partial sums (at most 32) and an addition (2) round off at most 2^-23, half of that and
2^-24 of S.  The 8-bit instruction, taken for results of 16 bits, also cuts each of the eight products that it adds at a
time off below 2^-13 of the largest, which costs the seven others less than 7 2^-13 of their group's magnitudes.  So
|z - exact| <= (8 K1 + 18) 2^-23 S in float32 and (2 K1 + 18) 2^-23 S + 7 2^-13 S in 16 bits; SiLU stretches that by at
most 1.1 and adds (|z| + 4) 2^-22 |y| for its exponential and division; then one rounding to the type.  The cut leaves
products of small integers whole, so on these every sum is exact and results are compared bit for bit.
"""
import ctypes

import numpy as np
import pytest
import torch

import convolution_int8_implicit_amd as ifx
from oracle import lowp
from test_mx4 import TYPES, excess, f64, note

FORMATS = {"e4m3": ifx.FP8_E4M3, "e5m2": ifx.FP8_E5M2}


def tensor_of(q, k, fmt=0, device="cuda"):
    return ifx.Fp8(torch.from_numpy(q[0].copy()).to(device), torch.from_numpy(q[1].copy()).to(device), k, fmt)


# ------------------------------------------------------------------------------------------ CPU

def test_reference_values_are_the_formats():
    """The 256 values of either format, against torch's own types; largest and smallest values by hand."""
    for fmt, dtype in ((0, torch.float8_e4m3fn), (1, torch.float8_e5m2)):
        t = torch.arange(256, dtype=torch.uint8).view(dtype).double().numpy()
        assert np.array_equal(lowp.FP8[fmt], t, equal_nan=True)
    assert lowp.FP8[0][0x7e] == 448 and lowp.FP8[0][1] == 2.0 ** -9 and np.isnan(lowp.FP8[0][0x7f])
    assert lowp.FP8[1][0x7b] == 57344 and lowp.FP8[1][1] == 2.0 ** -16 and np.isinf(lowp.FP8[1][0x7c])


def test_reference_rounding_pins():
    """Halves go to the even code, nothing saturates, the scale is the smallest that holds the largest magnitude."""
    x = np.zeros((1, 128))
    x[0, :8] = [448.0, 17.0, 19.0, 18.0, -27.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11]
    codes, scales = lowp.fp8_quantize(x)
    assert codes.shape == (1, 1, 128) and list(scales[0, 0]) == [127, 0, 0, 0]
    assert list(lowp.fp8_values(codes, scales, 128)[0, :8]) == [448, 16, 20, 18, -28, 0, 2.0 ** -8, 0]
    for fmt, most in ((0, 448.0), (1, 57344.0)):
        for e in (-140, -20, 0, 5, 100):
            for f, up in ((1.0, 0), (1 + 2.0 ** -20, 1), (0.999, 0), (1.0 / 1.75, 0)):
                top = most * f * 2.0 ** e
                s = int(lowp.fp8_quantize(np.array([[top]]), fmt)[1][0, 0, 0])
                assert s == max(0, 127 + e + up)
                assert top <= most * 2.0 ** (s - 127) and (s == 0 or top > most * 2.0 ** (s - 128))
    c, s = lowp.fp8_quantize(np.array([[1.0, np.inf], [np.nan, 0.0], [-0.0, 0.0]]))
    assert list(s[0, :, 0]) == [255, 255, 0] and not c[:, :2].any() and c[0, 2, 0] == 128


def test_reference_values_are_fixed_points():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 700)) * 10.0 ** rng.integers(-8, 8, (5, 700))
    for fmt, half in ((0, 2.0 ** -4), (1, 2.0 ** -3)):
        q = lowp.fp8_quantize(x, fmt)
        v = lowp.fp8_values(*q, 700, fmt)
        assert np.array_equal(lowp.fp8_values(*lowp.fp8_quantize(v, fmt), 700, fmt), v)
        unit = 2.0 ** (q[1].transpose(1, 0, 2).reshape(5, -1)[:, :6].astype(float) - 127).repeat(128, 1)[:, :700]
        assert (np.abs(v - x) <= np.maximum(half * np.abs(x), unit * lowp.FP8[fmt][1] / 2)).all()


def test_sizes_and_refusals_need_no_device():
    L = ifx.lib()
    fake, odd, half = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001), ctypes.c_void_p(0x100002)
    assert L.ifx_fp8_code_bytes(5, 129) == 2 * 5 * 128 and L.ifx_fp8_scale_bytes(5, 129) == 5 * 4
    assert L.ifx_fp8_scale_bytes(5, 512) == 5 * 4 and L.ifx_fp8_scale_bytes(5, 513) == 2 * 5 * 4
    assert L.ifx_fp8_code_bytes(-1, 5) == 0 and L.ifx_fp8_scale_bytes(1, 0) == 0
    for fn, args in ((L.ifx_fp8_quantize, lambda x, t, ld, r, k, c, s, f=0: (x, t, ld, r, k, f, c, s, None)),
                     (L.ifx_fp8_quantize_t, lambda x, t, ld, r, k, c, s, f=0: (x, t, ld, k, r, f, c, s, None)),
                     (L.ifx_fp8_dequantize, lambda x, t, ld, r, k, c, s, f=0: (c, s, f, r, k, x, t, ld, None))):
        turned = fn is L.ifx_fp8_quantize_t
        assert fn(*args(None, 0, 4, 1, 4, fake, fake)) == 1
        assert fn(*args(fake, 0, 4, 1, 4, None, fake)) == 1
        assert fn(*args(fake, 0, 4, 1, 4, fake, None)) == 1
        assert fn(*args(fake, 3, 4, 1, 4, fake, fake)) == 3
        assert fn(*args(fake, 0, 4, 1, 4, fake, fake, 2)) == 3
        assert fn(*args(fake, 0, 4, 1, 4, fake, fake, -1)) == 3
        assert fn(*args(fake, 0, 3, 1, 4, fake, fake)) == 2
        assert fn(*args(fake, 0, 4, -1, 4, fake, fake)) == 2
        assert fn(*args(fake, 0, 1 << 61, 4, 4, fake, fake)) == 2
        assert fn(*args(fake, 0, 1 << 30, (1 << 31) - 1, 1 << 30, fake, fake)) == 2
        assert fn(*args(half, 0, 4, 1, 4, fake, fake)) == 4
        assert fn(*args(odd, 1, 4, 1, 4, fake, fake)) == 4
        assert fn(*args(fake, 1, 4, 1, 4, ctypes.c_void_p(0x100008), fake)) == 4
        assert fn(*args(fake, 1, 4, 1, 4, fake, half)) == 4
        # nothing to do for no rows of the result; no columns are refused
        assert fn(*args(None, 1, 4, *((4, 0) if turned else (0, 4)), None, None)) == 0
        assert fn(*args(fake, 0, 4, *((0, 4) if turned else (1, 0)), fake, fake)) == 2
    # a transposed launch: of panels by 32 columns
    assert L.ifx_fp8_quantize_t(fake, 0, 1 << 28, 1 << 28, 1 << 9, 0, fake, fake, None) == 2
    assert L.ifx_fp8_quantize_t(fake, 1, (1 << 31) - 1, (1 << 31) - 1, 1, 0, fake, fake, None) == 2

    def mm(m=2, n=3, k=4, f=0, t=1, act=0, ld_y=3, ld_res=3, a=fake, asc=fake, w=fake, wsc=fake, bias=fake, res=fake, y=fake):
        return L.ifx_fp8_matmul(ctypes.byref(ifx.Fp8Desc(m, n, k, f, t, act, ld_y, ld_res)), a, asc, w, wsc, bias, res, y,
                                None)
    assert L.ifx_fp8_matmul(None, fake, fake, fake, fake, None, None, fake, None) == 1
    for name in ("a", "asc", "w", "wsc", "y"):
        assert mm(**{name: None}) == 1, name
    assert mm(t=5) == 3 and mm(act=3) == 3 and mm(act=-1) == 3 and mm(f=2) == 3
    assert mm(m=-1) == 2 and mm(n=-1) == 2 and mm(k=0) == 2 and mm(ld_y=2) == 2 and mm(ld_res=2) == 2
    assert mm(y=odd) == 4 and mm(res=odd) == 4 and mm(bias=half) == 4 and mm(a=half) == 4 and mm(wsc=half) == 4
    assert mm(m=0, a=None, y=None) == 0 and mm(n=0, ld_y=0, ld_res=0, w=None) == 0
    assert mm(m=1 << 18, n=1 << 17, ld_y=1 << 17, ld_res=1 << 17, y=None) == 1
    assert mm(m=1 << 18, n=1 << 18, ld_y=1 << 18, ld_res=1 << 18) == 2


def test_binding_refusals_need_no_device(monkeypatch):
    x = torch.zeros(4, 32)
    for call in (ifx.fp8_quantize, ifx.fp8_quantize_t):
        with pytest.raises(ValueError):
            call(x)  # not on a GPU
    monkeypatch.setattr(ifx, "_on_device", lambda *ts: 0)
    monkeypatch.setattr(ifx, "_raw_stream", lambda stream, index: 0)

    def fp8(rows, k, fmt=0):
        return ifx.fp8_empty(rows, k, fmt, device="meta")
    with pytest.raises(ValueError):
        ifx._fp8_check(ifx.Fp8(torch.zeros(1, 4, 128, dtype=torch.uint8), torch.zeros(1, 3, 4, dtype=torch.uint8), 32), "a")
    with pytest.raises(ValueError):
        ifx._fp8_check(ifx.Fp8(torch.zeros(1, 4, 128, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8), 129), "a")
    x = torch.empty(4, 32, device="meta")
    for out in (fp8(5, 32), fp8(4, 33), fp8(4, 32, 1)):
        with pytest.raises(ValueError):
            ifx.fp8_quantize(x, out=out)
    with pytest.raises(ValueError):
        ifx.fp8_quantize_t(x, out=fp8(4, 32))
    with pytest.raises(ValueError):
        ifx.fp8_quantize(x.t())
    with pytest.raises(TypeError):
        ifx.fp8_quantize(torch.empty(4, 32, device="meta", dtype=torch.int8))
    with pytest.raises(ValueError):
        ifx.fp8_matmul(fp8(4, 32), fp8(4, 33))
    with pytest.raises(ValueError, match="E4M3"):
        ifx.fp8_matmul(fp8(4, 32), fp8(4, 32, 1))
    with pytest.raises(ValueError):
        ifx.fp8_matmul(fp8(4, 32), fp8(5, 32), bias=torch.empty(4, device="meta"))
    with pytest.raises(ValueError):
        ifx.fp8_matmul(fp8(4, 32), fp8(5, 32), residual=torch.empty(4, 5, device="meta"))
    with pytest.raises(ValueError):
        ifx.fp8_matmul(fp8(4, 32), fp8(5, 32), out=torch.empty(5, 4, device="meta"))
    # sizes past 32 bits are refused by the binding, not taken modulo 2^32
    big, fit = (1 << 32) + 5, 5
    for call in (lambda b: ifx.fp8_quantize(torch.empty(b, 3, device="meta")),
                 lambda b: ifx.fp8_quantize(torch.empty(3, b, device="meta")),
                 lambda b: ifx.fp8_quantize_t(torch.empty(b, 3, device="meta")),
                 lambda b: ifx.fp8_quantize_t(torch.empty(3, b, device="meta")),
                 lambda b: ifx.fp8_dequantize(fp8(b, 3)), lambda b: ifx.fp8_dequantize(fp8(3, b)),
                 lambda b: ifx.fp8_matmul(fp8(b, 3), fp8(4, 3)), lambda b: ifx.fp8_matmul(fp8(4, 3), fp8(b, 3)),
                 lambda b: ifx.fp8_matmul(fp8(4, b), fp8(4, b)), lambda b: ifx.fp8_matmul(fp8(4, 3), fp8(4, 3), act=b - fit)):
        with pytest.raises(ifx.IfxError, match="NULL"):
            call(fit)
        with pytest.raises(ValueError, match="32 bits"):
            call(big)


# ------------------------------------------------------------------------------------------ GPU

def block_values(rows, k, kind, seed):
    """Values of every magnitude that the type holds, among them zeros, exact halves between codes, block maxima at
    and around the formats' largest values, subnormals, the type's extremes, infinities and NaN (one block each)."""
    rng = np.random.default_rng(seed)
    low, high = {"f32": (-148, 126), "bf16": (-132, 126), "f16": (-23, 13)}[kind]
    x = rng.standard_normal((rows, k)) * 2.0 ** rng.integers(low + 12, high, (rows, 1))
    pick = rng.random((rows, k))
    unit = 2.0 ** rng.integers(low + 3, high - 9, (rows, 1))
    near = rng.choice([0, .5, 1, 1.5, 2.5, 17, 18, 19, 27, 29, 36, 44, 104, 112, 120, 416, 432, 448, 449, 464], (rows, k))
    x = np.where(pick < 0.3, unit * near * rng.choice([-1, 1], (rows, k)), x)
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


def same_codes(q, expect):
    return np.array_equal(q.scales.cpu().numpy(), expect[1]) and np.array_equal(q.codes.cpu().numpy(), expect[0])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 2048), (7, 31), (5, 127), (17, 128), (33, 130), (16, 515), (50, 997)])
def test_quantize(rows, k, kind):
    x = block_values(rows, k, kind, 7 * rows + k)
    for fmt in (0, 1):
        note(f"quantize {rows} x {k} {kind} format {fmt}")
        expect = lowp.fp8_quantize(f64(x), fmt)
        q = ifx.fp8_quantize(x.cuda(), fmt)
        assert q.format == fmt and q.rows == rows and same_codes(q, expect)
        v = lowp.fp8_values(*expect, k, fmt)
        for dtype in (torch.float32, torch.bfloat16, torch.float16):
            with np.errstate(over="ignore", invalid="ignore"):
                rounded = v.astype(np.float16).astype(np.float64) if dtype == torch.float16 else v
            got = ifx.fp8_dequantize(q, dtype)
            assert got.shape == (rows, k) and got.dtype == dtype
            # (bfloat16 holds four bits of any value of 2^-126 and more, and those of e4m3 down to 2^-133)
            if dtype == torch.bfloat16:
                rounded = f64(torch.from_numpy(v).to(torch.bfloat16))
            if dtype == torch.float32:
                rounded = v.astype(np.float32).astype(np.float64)
            assert np.array_equal(f64(got), rounded, equal_nan=True)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("k,n", [(1, 1), (1, 70), (31, 7), (127, 5), (128, 64), (130, 33), (515, 16), (997, 131)])
def test_quantize_transposed(k, n, kind):
    """The codes of the transpose, also of a slice at an odd offset."""
    x = block_values(k, n, kind, 3 * k + n)
    for fmt in (0, 1):
        note(f"quantize_t {k} x {n} {kind} format {fmt}")
        expect = lowp.fp8_quantize(f64(x).T, fmt)
        q = ifx.fp8_quantize_t(x.cuda(), fmt)
        assert q.rows == n and q.k == k and same_codes(q, expect)
    wide = torch.full((k, n + 9), float("nan"), dtype=TYPES[kind], device="cuda")
    wide[:, 3:3 + n] = x.cuda()
    out = ifx.fp8_empty(n, k, 1)
    out.codes.fill_(0xAA)
    out.scales.fill_(0xAA)
    assert ifx.fp8_quantize_t(wide[:, 3:3 + n], 1, out=out) is out and same_codes(out, expect)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
def test_every_code_and_every_float16(fmt):
    """Every code's value, under scales from 0 to 254 and NaN; every finite float16 beside a larger one."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(2, 1, 128).expand(2, 256, 128).contiguous()
    scales = torch.zeros(1, 256, 4, dtype=torch.uint8, device="cuda")
    scales[0, :, :2] = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None]
    q = ifx.Fp8(codes, scales, 256, fmt)
    with np.errstate(over="ignore"):
        v = lowp.fp8_values(codes.cpu().numpy(), scales.cpu().numpy(), 256, fmt).astype(np.float32)
    assert np.array_equal(ifx.fp8_dequantize(q, torch.float32).cpu().numpy(), v, equal_nan=True)
    h = np.arange(65536, dtype=np.uint16).view(np.float16)
    h = h[np.isfinite(h)]
    x = np.zeros((h.size, 130), dtype=np.float16)
    x[:, 0], x[:, 5], x[:, 127] = h, h / np.float16(16), h * np.float16(0.5625)
    x[:, 129] = h
    assert same_codes(ifx.fp8_quantize(torch.from_numpy(x).cuda(), fmt), lowp.fp8_quantize(x, fmt))


@pytest.mark.gpu
def test_quantize_strides_streams_and_out():
    """A slice of a wider tensor at an odd offset, more axes than two, another stream, given outputs."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(3, 5, 7, 301, device="cuda", generator=gen).to(torch.bfloat16)
    x = wide[..., 3:300]
    expect = lowp.fp8_quantize(f64(x).reshape(-1, 297))
    out = ifx.fp8_empty(105, 297)
    out.codes.fill_(0xAA)
    out.scales.fill_(0xAA)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = ifx.fp8_quantize(x, out=out, stream=s)
    t = ifx.fp8_quantize_t(x, stream=s)
    dst = torch.full((105, 400), 7.0, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    ifx.fp8_dequantize(q, out=dst[:, 1:298], stream=s.cuda_stream)
    s.synchronize()
    assert q.codes is out.codes and same_codes(out, expect)
    assert same_codes(t, lowp.fp8_quantize(f64(x).reshape(-1, 297).T))
    assert np.array_equal(f64(dst[:, 1:298]), lowp.fp8_values(*expect, 297))
    assert (dst[:, 0] == 7).all() and (dst[:, 298:] == 7).all()


@pytest.mark.gpu
def test_empty_and_refusals():
    q = ifx.fp8_quantize(torch.empty(0, 64, device="cuda"))
    assert q.codes.shape == (1, 0, 128) and ifx.fp8_dequantize(q).shape == (0, 64)
    assert ifx.fp8_quantize_t(torch.empty(64, 0, device="cuda")).codes.shape == (1, 0, 128)
    w = ifx.fp8_quantize(torch.ones(6, 64, device="cuda"))
    assert ifx.fp8_matmul(q, w).shape == (0, 6) and ifx.fp8_matmul(w, q).shape == (6, 0)
    with pytest.raises(ifx.IfxError):
        ifx.fp8_quantize(torch.empty(4, 0, device="cuda"))
    with pytest.raises(ifx.IfxError):
        ifx.fp8_quantize_t(torch.empty(0, 4, device="cuda"))
    with pytest.raises(ifx.IfxError):
        ifx.fp8_matmul(w, w, act=9)
    with pytest.raises(ValueError):
        ifx.fp8_matmul(w, w, residual=torch.ones(6, 6, device="cuda", dtype=torch.bfloat16).t())


def random_codes(rng, rows, k, fmt=0, low=118, high=134):
    """Codes over all finite values, one row of zeros, scales of a few powers of two; zeros past k."""
    k1 = (k + 127) // 128
    codes = rng.integers(0, 256, (k1, rows, 128), dtype=np.uint8)
    codes = np.where(codes & 127 > (0x7b if fmt else 0x7e), codes & 0xf0, codes)
    codes[np.broadcast_to(np.arange(k1 * 128).reshape(k1, 1, 128) >= k, codes.shape)] = 0
    scales = np.zeros(((k1 + 3) // 4, rows, 4), dtype=np.uint8)
    flat = rng.integers(low, high, (rows, k1))
    scales.transpose(1, 0, 2).reshape(rows, -1)
    full = np.zeros((rows, (k1 + 3) // 4 * 4), dtype=np.uint8)
    full[:, :k1] = flat
    scales = np.ascontiguousarray(full.reshape(rows, -1, 4).transpose(1, 0, 2))
    if rows > 2:
        codes[:, 1] = 0
    return codes.astype(np.uint8), scales


def product_case(m, n, k, seed, fmt=0):
    rng = np.random.default_rng(seed)
    # products of about 2^0: e4m3 codes reach 2^8, e5m2 2^15
    a = random_codes(rng, m, k, fmt, 112 if fmt else 118, 118 if fmt else 124)
    w = random_codes(rng, n, k, 0, 118, 124)
    return a, w, rng.standard_normal(n).astype(np.float32) * 30, rng.standard_normal((m, n)) * 30


def sum_bound(k, kind):
    """How far a sum of k products is off, of the sum of their magnitudes."""
    k1 = (k + 127) // 128
    return (8 * k1 + 18) * 2.0 ** -23 if kind == "f32" else (2 * k1 + 18) * 2.0 ** -23 + 7 * 2.0 ** -13


def check_product(y, m, n, k, a, w, bias, res, act, kind, fmt=0):
    exact, z, s = lowp.fp8_matmul(a, w, k, fmt, bias, res, act)
    tol = sum_bound(k, kind) * s
    if act == ifx.ACT_SILU:
        tol = 1.1 * tol + (np.abs(z) + 4) * 2.0 ** -22 * np.abs(exact)
    got = f64(y)
    assert got.shape == (m, n)
    assert (np.isnan(got) == np.isnan(exact)).all()
    assert excess(got, exact, tol, kind) == 0


SHAPES = [(1, 1, 1), (1, 40, 2048), (1, 33, 4224), (2, 17, 33), (3, 50, 4100), (5, 1000, 130), (7, 60, 2200), (16, 16, 128),
          (17, 31, 129), (33, 65, 640), (64, 64, 256), (65, 130, 96), (100, 300, 1000), (130, 257, 385), (257, 129, 512),
          (300, 520, 64),
          # enough tiles for the larger ones, edges inside a tile, one to nine steps of the ring
          (1000, 1500, 200), (1900, 1700, 700), (2050, 2049, 300), (2111, 1930, 1100), (4097, 4100, 130), (4200, 3970, 600)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul(m, n, k):
    for i, (kind, act) in enumerate((("f32", 0), ("bf16", 1), ("f16", 2))):
        if i and m * n > 10_000_000:
            continue
        fmt = (i + m) % 2
        note(f"product {m} x {n} x {k} {kind} format {fmt}")
        a, w, bias, res = product_case(m, n, k, m + 3 * n + 7 * k, fmt)
        b = bias if i != 1 or m % 2 else None
        r = torch.from_numpy(res).to(TYPES[kind]) if (i + n) % 2 else None
        if kind == "f16":  # keeps float16 results finite
            a = (a[0], a[1] - 6 * (a[1] > 0).astype(np.uint8))
        y = ifx.fp8_matmul(tensor_of(a, k, fmt), tensor_of(w, k), None if b is None else torch.from_numpy(b).cuda(),
                           None if r is None else r.cuda(), act, TYPES[kind])
        check_product(y, m, n, k, a, w, b, None if r is None else f64(r), act, kind, fmt)


def integer_codes(rng, rows, k, fmt=0, most=3):
    """e4m3 or e5m2 codes of whole numbers up to `most` in magnitude, every scale 1."""
    x = rng.integers(-most, most + 1, (rows, k)).astype(np.float64)
    table = lowp.FP8[fmt]
    codes = np.array([int(np.argmax(table == v)) for v in range(most + 1)], dtype=np.uint8)
    k1 = (k + 127) // 128
    c = np.zeros((rows, k1 * 128), dtype=np.uint8)
    c[:, :k] = codes[np.abs(x).astype(int)] + 128 * (x < 0)
    s = np.zeros((rows, (k1 + 3) // 4 * 4), dtype=np.uint8)
    s[:, :k1] = 127
    return (np.ascontiguousarray(c.reshape(rows, k1, 128).transpose(1, 0, 2)),
            np.ascontiguousarray(s.reshape(rows, -1, 4).transpose(1, 0, 2)))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul_of_whole_numbers(m, n, k):
    """Sums that every step leaves exact: results are those of whole numbers, rounded once, whatever kernel runs."""
    rng = np.random.default_rng(m * n + k)
    for kind in ("bf16", "f16", "f32"):
        for fmt in (0, 1):
            if m * n > 4_000_000 and fmt:
                continue
            note(f"whole numbers {m} x {n} x {k} {kind} format {fmt}")
            a, w = integer_codes(rng, m, k, fmt), integer_codes(rng, n, k)
            exact = lowp.fp8_values(*a, k, fmt) @ lowp.fp8_values(*w, k).T
            y = ifx.fp8_matmul(tensor_of(a, k, fmt), tensor_of(w, k), dtype=TYPES[kind])
            assert torch.equal(y.cpu(), torch.from_numpy(exact).to(TYPES[kind]))


@pytest.mark.gpu
def test_matmul_error_on_normal_values():
    """On normally distributed values: float32 results within a few roundings, 16-bit ones within theirs."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    for m in (16, 300):
        a = ifx.fp8_quantize(torch.randn(m, 4096, device="cuda", generator=gen))
        w = ifx.fp8_quantize(torch.randn(500, 4096, device="cuda", generator=gen))
        exact = f64(ifx.fp8_dequantize(a, torch.float32)) @ f64(ifx.fp8_dequantize(w, torch.float32)).T
        # a rounding's error is uniform within half a step, so less than 2^-9 / sqrt(3) and 2^-12 / sqrt(3) of a value
        for kind, most in (("f32", 2.0 ** -20), ("bf16", 2.0 ** -9), ("f16", 2.0 ** -12)):
            err = f64(ifx.fp8_matmul(a, w, dtype=TYPES[kind])) - exact
            assert np.linalg.norm(err) <= most * np.linalg.norm(exact), (m, kind)


@pytest.mark.gpu
def test_matmul_long_sums():
    """Every step of the large tile's ring many times over, ragged edges; rows sampled."""
    m, n, k = 4100, 4090, 4200
    a, w, bias, res = product_case(m, n, k, 77)
    rows = np.unique(np.r_[0:3, 255:258, 2047:2050, m - 5:m, np.random.default_rng(2).integers(0, m, 40)])
    some = tuple(np.ascontiguousarray(t[:, rows]) for t in a)
    for kind, act in (("f32", 0), ("bf16", 1)):
        note(f"product {m} x {n} x {k} {kind}")
        r = torch.from_numpy(res).to(TYPES[kind])
        y = ifx.fp8_matmul(tensor_of(a, k), tensor_of(w, k), torch.from_numpy(bias).cuda(), r.cuda(), act, TYPES[kind])
        check_product(y[torch.from_numpy(rows).cuda()], len(rows), n, k, some, w, bias, f64(r)[rows], act, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 6, 40, 300])
def test_matmul_nan_blocks_and_extreme_scales(m):
    """A NaN scale or code spoils its row or column alone; scales far apart multiply exactly."""
    n, k = 70, 2300
    note(f"product with NaN blocks, m = {m}")
    a, w, _, _ = product_case(m, n, k, 11 + m)
    w[1][1, 5, 2] = 255
    w[1][4, n - 1, 1] = 255
    w[0][3, 9, 17] = 0x7f
    nan = np.zeros((m, n), dtype=bool)
    nan[:, [5, 9, n - 1]] = True
    if m > 3:
        a[1][0, 3, 1] = 255
        a[0][2, 4, 100] = 0xff
        nan[3:5] = True
    y = f64(ifx.fp8_matmul(tensor_of(a, k), tensor_of(w, k), dtype=torch.float32))
    assert (np.isnan(y) == nan).all()
    check_product(torch.from_numpy(y), m, n, k, a, w, None, None, 0, "f32")
    for q, byte in ((a, 238), (w, 16)):
        some = q[1] > 0
        q[1][some] = byte
    for kind in ("f32", "bf16"):
        check_product(ifx.fp8_matmul(tensor_of(a, k), tensor_of(w, k), dtype=TYPES[kind]), m, n, k, a, w, None, None, 0, kind)


@pytest.mark.gpu
def test_infinities_of_e5m2():
    """An infinity of e5m2 in A gives infinities, or NaN against a zero."""
    a, w, _, _ = product_case(70, 40, 200, 5, 1)
    a[0][1, 3, 7] = 0x7c
    w[0][1, 5, 7] = 0
    w[0][1, 6, 7] = 0x38
    y = f64(ifx.fp8_matmul(tensor_of(a, 200, 1), tensor_of(w, 200), dtype=torch.float32))
    assert not np.isfinite(y[3]).any() and np.isnan(y[3, 5]) and y[3, 6] == np.inf
    assert np.isfinite(np.delete(y, 3, 0)).all()


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
        got = ifx.fp8_matmul(A, W, B, y, ifx.ACT_RELU, out=y, stream=s)
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
    a = (a[0], a[1] - 5 * (a[1] > 0).astype(np.uint8))  # keeps float16 results finite
    for kind, with_res in (("bf16", False), ("f16", True), ("f32", True)):
        note(f"product {m} x {n} x {k} {kind}, rows of {pitch}")
        r = torch.from_numpy(res).to(TYPES[kind]) if with_res else None
        wide = torch.full((m, pitch), 3.0, dtype=TYPES[kind], device="cuda")
        ifx.fp8_matmul(tensor_of(a, k), tensor_of(w, k), torch.from_numpy(bias).cuda(), None if r is None else r.cuda(),
                       ifx.ACT_RELU, out=wide[:, :n])
        check_product(wide[:, :n], m, n, k, a, w, bias, None if r is None else f64(r), ifx.ACT_RELU, kind)
        assert bool((wide[:, n:] == 3).all())
    codes, scales = random_codes(np.random.default_rng(3), m, 117)
    v = lowp.fp8_values(codes, scales, 117)
    for kind in ("bf16", "f16", "f32"):
        note(f"values {m} x 117 {kind}, rows of {pitch}")
        wide = torch.full((m, pitch), 3.0, dtype=TYPES[kind], device="cuda")
        ifx.fp8_dequantize(tensor_of((codes, scales), 117), out=wide[:, :117])
        assert np.array_equal(f64(wide[:, :117]), v.astype(np.float16).astype(np.float64) if kind == "f16" else v)
        assert bool((wide[:, 117:] == 3).all())


@pytest.mark.gpu
@pytest.mark.parametrize("m", [2, 130])
def test_matmul_same_from_call_to_call_and_in_a_graph(m):
    n, k = 200, 4096
    a, w, bias, _ = product_case(m, n, k, 9)
    A, W, B = tensor_of(a, k), tensor_of(w, k), torch.from_numpy(bias).cuda()
    first = ifx.fp8_matmul(A, W, B)
    out = torch.empty_like(first)
    x = torch.randn(m, k, device="cuda")
    q, t = ifx.fp8_empty(m, k), ifx.fp8_empty(k, m)
    ifx.fp8_quantize(x, out=q)
    ifx.fp8_quantize_t(x, out=t)
    other = ifx.fp8_matmul(q, W, B)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ifx.fp8_quantize(x, out=q)
        ifx.fp8_quantize_t(x, out=t)
        ifx.fp8_matmul(q, W, B, out=out)
    for i in range(4):
        q.codes.zero_()
        t.codes.zero_()
        out.zero_()
        x.add_(0.0 if i < 2 else 1.0)
        g.replay()
        expect, turned = ifx.fp8_matmul(ifx.fp8_quantize(x), W, B), ifx.fp8_quantize_t(x)
        torch.cuda.synchronize()
        assert torch.equal(out, expect) and torch.equal(t.codes, turned.codes) and torch.equal(t.scales, turned.scales)
        if i < 2:
            assert torch.equal(out, other)
        assert torch.equal(ifx.fp8_matmul(A, W, B), first)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,n,k,kind", [(6241, 50, 70, "f32"), (900, 300, 257, "bf16"), (1, 40, 33, "f16")])
def test_weight_gradient(tokens, n, k, kind):
    """dy^T x from the tensors themselves: rounding of both transposes, dy to e5m2, and the product."""
    note(f"weight gradient {n} x {k} of {tokens} tokens, {kind}")
    gen = torch.Generator().manual_seed(tokens)
    dy = (torch.randn(tokens, n, generator=gen) / 100).to(TYPES[kind])
    x = torch.randn(tokens, k, generator=gen).to(TYPES[kind])
    dw = ifx.fp8_matmul(ifx.fp8_quantize_t(dy.cuda(), ifx.FP8_E5M2), ifx.fp8_quantize_t(x.cuda()), dtype=torch.float32)
    a, w = lowp.fp8_quantize(f64(dy).T, 1), lowp.fp8_quantize(f64(x).T)
    check_product(dw, n, k, tokens, a, w, None, None, 0, "f32", 1)
    # of the gradient in 64 bits, every operand rounded once: 2^-3 and 2^-4 of a value (and below a block's 2^-16 or
    # 2^-9 units half of that) at most
    err = np.abs(f64(dw) - f64(dy).T @ f64(x))
    assert (err <= (2.0 ** -3 + 2.0 ** -4 + 2.0 ** -7 + 2.0 ** -8) * (np.abs(f64(dy)).T @ np.abs(f64(x))) +
            2.0 ** -15 * np.abs(f64(dy)).max() * np.abs(f64(x)).sum(0) + 2.0 ** -9 * np.abs(f64(x)).max() * np.abs(f64(dy)).sum(0)[:, None]).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^32 bytes and 2^31 elements, and codes past 2^32 bytes."""
    rows, k = (1 << 21) + 5, 1100
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(37, k, device="cuda", generator=gen)
    x[-37:] = tail
    note("rounding")
    q = ifx.fp8_quantize(x)
    codes, scales = lowp.fp8_quantize(f64(x[-37:]))
    assert np.array_equal(q.codes[:, -37:].cpu().numpy(), codes) and np.array_equal(q.scales[:, -37:].cpu().numpy(), scales)
    assert not q.codes[:, :-37].any()
    v = ifx.fp8_dequantize(q)
    assert np.array_equal(f64(v[-37:]), lowp.fp8_values(codes, scales, k)) and not v[:-37].any()
    del v, q
    note("rounding of the transpose")
    t = ifx.fp8_quantize_t(x)
    last = rows // 128 * 128
    codes, scales = lowp.fp8_quantize(f64(x[last - 128:]).T)
    assert np.array_equal(t.codes[-2:].cpu().numpy(), codes) and not t.codes[:-2].any()
    s = t.scales.permute(1, 0, 2).reshape(k, -1)[:, rows // 128 - 1:rows // 128 + 1].cpu().numpy()
    assert np.array_equal(s, scales[0, :, :2])
    del x, t
    note("product")
    m, k = (1 << 20) + 3, 4096 + 128
    a = ifx.fp8_empty(m, k)
    a.codes.zero_()
    a.scales.zero_()
    assert a.codes.numel() > 1 << 32
    t = ifx.fp8_quantize(torch.randn(40, k, device="cuda", generator=gen))
    a.codes[:, -40:], a.scales[:, -40:] = t.codes, t.scales
    w = ifx.fp8_quantize(torch.randn(24, k, device="cuda", generator=gen))
    y = ifx.fp8_matmul(a, w)
    few = (t.codes.cpu().numpy(), t.scales.cpu().numpy())
    check_product(y[-40:], 40, 24, k, few, (w.codes.cpu().numpy(), w.scales.cpu().numpy()), None, None, 0, "bf16")
    assert not y[:-40].any()


def whole_excess(got, exact, tol, kind):
    """excess() of whole large results, on the GPU."""
    low, high = ((exact + sign * tol).to(TYPES[kind]).double() for sign in (-1, 1))
    out = torch.maximum(low - got.double(), got.double() - high).clamp_(min=0)
    return float(out.max()) if not bool(out.isnan().any()) else np.inf


def cuda64(q, k, fmt=0):
    return torch.from_numpy(np.ascontiguousarray(lowp.fp8_values(q[0], q[1], k, fmt))).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kind,fmt", [("bf16", 0), ("bf16", 1), ("f16", 0), ("f16", 1), ("f32", 0), ("f32", 1)])
@pytest.mark.parametrize("extra", [0, 64, 3])
def test_matmul_many_large_tiles(kind, fmt, extra):
    """Large tiles of either format of A and every type: the ring refilled many times, three words of scales, whole tiles
    and edges inside a tile, results past the caches' size in rows that fill 128-byte lines (extra 0 and 64) and rows
    that share them; bias and residual in turn.  Every result is checked, and what lies beside the rows."""
    m, n, k = 4200, 4160, 1200
    note(f"large tiles {m} x {n} x {k} {kind} format {fmt}, rows of {n + extra}")
    rng = np.random.default_rng(21 + fmt)
    a, w = random_codes(rng, m, k, fmt, 112 if fmt else 118, 118 if fmt else 124), random_codes(rng, n, k, 0, 118, 124)
    if kind == "f16":  # keeps float16 results finite
        a = (a[0], a[1] - 6 * (a[1] > 0).astype(np.uint8))
    gen = torch.Generator(device="cuda").manual_seed(3)
    bias = torch.randn(n, generator=gen, device="cuda") * 30
    res = (torch.randn(m, n, generator=gen, device="cuda") * 30).to(TYPES[kind])
    av, wv = cuda64(a, k, fmt), cuda64(w, k)
    z, size = av @ wv.t(), av.abs() @ wv.abs().t()
    A, W = tensor_of(a, k, fmt), tensor_of(w, k)
    for b, r in ((bias, None), (None, res)):
        wide = torch.full((m, n + extra), 3.0, dtype=TYPES[kind], device="cuda")
        ifx.fp8_matmul(A, W, b, r, ifx.ACT_NONE, out=wide[:, :n])
        term = (b if r is None else r).double()
        assert whole_excess(wide[:, :n], z + term, sum_bound(k, kind) * (size + term.abs()), kind) == 0
        assert bool((wide[:, n:] == 3).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", [(6, 40), (70, 40), (300, 520), (4100, 4100)])
def test_infinities_of_e5m2_in_every_kernel(m, n, kind):
    """An infinity of e5m2 gives infinities of its sign and W's, or NaN against a zero or a NaN, in its row alone."""
    note(f"an infinity in {m} x {n} {kind}")
    k = 200
    rng = np.random.default_rng(m + n)
    a, w = integer_codes(rng, m, k, 1), integer_codes(rng, n, k)
    for row, code in ((3, 0x7c), (m - 1, 0xfc)):
        a[0][1, row, 7] = code
    w[0][1, :, 7] = 0x38  # 1
    w[0][1, 5, 7], w[0][1, 6, 7], w[0][1, n - 1, 7] = 0, 0xb8, 0xb8
    y = f64(ifx.fp8_matmul(tensor_of(a, k, 1), tensor_of(w, k), dtype=TYPES[kind]))
    expect = np.full(n, np.inf)
    expect[5], expect[6], expect[n - 1] = np.nan, -np.inf, -np.inf
    assert np.array_equal(y[3], expect, equal_nan=True) and np.array_equal(y[m - 1], -expect, equal_nan=True)
    rest = np.delete(np.arange(m), [3, m - 1])
    av = torch.from_numpy(lowp.fp8_values(a[0][:, rest], a[1][:, rest], k, 1))
    exact = av @ torch.from_numpy(lowp.fp8_values(*w, k)).t()
    assert np.array_equal(y[rest], f64(exact.to(TYPES[kind])))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 6, 40, 300])
@pytest.mark.parametrize("fmt,byte", [(0, 247), (1, 240)])
def test_matmul_largest_scales(m, fmt, byte):
    """The largest scales that a rounding gives.  Codes whose value float32 holds multiply exactly; one of 2^128 is finite
    in a 16-bit result, whose matrix instruction adds exponents, and infinite in float32, whose operands are widened."""
    n, k = 70, 700
    note(f"scale {byte} of format {fmt}, {m} rows")
    a, w, _, _ = product_case(m, n, k, 31 + m, fmt)
    a[1][a[1] > 0] = byte
    w[1][w[1] > 0] = 16
    a[0][(a[0] & 127) >= 0x78] &= 0x83  # from 256 (32768) on
    for kind in ("f32", "bf16"):
        check_product(ifx.fp8_matmul(tensor_of(a, k, fmt), tensor_of(w, k), dtype=TYPES[kind]), m, n, k, a, w, None, None, 0,
                      kind, fmt)
    a[0][1, m - 1, 3] = 0x78  # 256 2^120 or 32768 2^113
    w[0][1, 3, 3], w[0][1, 4, 3], w[0][1, 5, 3] = 0x38, 0xb8, 0
    A, W = tensor_of(a, k, fmt), tensor_of(w, k)
    check_product(ifx.fp8_matmul(A, W, dtype=torch.bfloat16), m, n, k, a, w, None, None, 0, "bf16", fmt)
    y = f64(ifx.fp8_matmul(A, W, dtype=torch.float32))
    assert y[m - 1, 3] == np.inf and y[m - 1, 4] == -np.inf and np.isnan(y[m - 1, 5])
    assert np.isfinite(y[:m - 1]).all()
    # such a value comes of a rounding: of the largest float32
    q = ifx.fp8_quantize(torch.full((1, 1), torch.finfo(torch.float32).max, device="cuda"), fmt)
    assert int(q.scales[0, 0, 0]) == byte and int(q.codes[0, 0, 0]) == 0x78 and bool(ifx.fp8_dequantize(q, torch.float32).isinf())
