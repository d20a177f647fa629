"""Plain 64-bit reference of the 4-bit, 8-bit and norm operators (numpy, CPU), written from their
formulas and sharing no code with the library.

A microscaled tensor of `rows` rows and k columns: blocks of 32 columns, codes of 4 bits (magnitudes 0, 0.5,
1, 1.5, 2, 3, 4, 6 and a sign) and a power of two 2^(s - 127) per block; codes [K1, rows, 64] bytes, scales
[K1, rows, 4] bytes, K1 = ceil(k / 128).

An 8-bit tensor: blocks of 128 columns, one byte a column (format 0: sign, four exponent and three mantissa bits, no
infinity; 1: sign, five and two) and a power of two 2^(s - 127) per block; codes [K1, rows, 128] bytes, scales
[ceil(K1 / 4), rows, 4] bytes.
"""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quantize(x: np.ndarray):
    """Codes and scales of x [rows, k] (any float type; exact in float64)."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    k1 = (k + 127) // 128
    b = np.zeros((rows, k1 * 128))
    b[:, :k] = x
    b = b.reshape(rows, k1 * 4, 32)
    codes = np.zeros(b.shape, dtype=np.uint8)
    scales = np.zeros(b.shape[:2], dtype=np.uint8)
    for r in range(rows):
        for j in range(k1 * 4):
            block = b[r, j]
            if not np.all(np.isfinite(block)):
                scales[r, j] = 255
                continue
            top = np.max(np.abs(block))
            s = max(0, int(np.frexp(top)[1]) - 1 + 125) if top > 0 else 0
            scales[r, j] = s
            unit = np.ldexp(np.abs(block), 127 - s)
            far = np.abs(unit[:, None] - LEVELS[None, :])
            near = far == far.min(axis=1, keepdims=True)
            # of two levels as near, the even code
            c = np.where(near.sum(axis=1) == 1, near.argmax(axis=1),
                         np.where(near.argmax(axis=1) % 2 == 0, near.argmax(axis=1), near.argmax(axis=1) + 1))
            codes[r, j] = c + 8 * np.signbit(block)
    packed = codes.reshape(rows, k1, 64, 2)
    packed = (packed[..., 0] + 16 * packed[..., 1]).astype(np.uint8).transpose(1, 0, 2)
    return np.ascontiguousarray(packed), np.ascontiguousarray(scales.reshape(rows, k1, 4).transpose(1, 0, 2))


def mx4_values(codes: np.ndarray, scales: np.ndarray, k: int) -> np.ndarray:
    """float64 [rows, k]: the values that codes and scales stand for."""
    k1, rows, _ = codes.shape
    c = np.stack((codes & 15, codes >> 4), -1).reshape(k1, rows, 4, 32)
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = scales.astype(np.int64)
    v = np.ldexp(v, (s - 127)[..., None])
    v[s == 255] = np.nan
    return v.reshape(k1, rows, 128).transpose(1, 0, 2).reshape(rows, k1 * 128)[:, :k]


def act(z: np.ndarray, kind: int) -> np.ndarray:
    if kind == 1:
        return np.where(z < 0, 0.0, z)
    if kind == 2:
        with np.errstate(over="ignore"):
            return z / (1 + np.exp(-z))
    return z


def act_grad(z: np.ndarray, kind: int) -> np.ndarray:
    if kind == 1:
        return (z > 0).astype(np.float64)
    if kind == 2:
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def mx4_matmul(a, w, k: int, bias=None, residual=None, kind: int = 0):
    """(y, z, s): the product after the activation, before it, and the sum of its terms' magnitudes."""
    av, wv = mx4_values(*a, k), mx4_values(*w, k)
    z, s = av @ wv.T, np.abs(av) @ np.abs(wv).T
    for term in (bias, residual):
        if term is not None:
            z, s = z + np.asarray(term, dtype=np.float64), s + np.abs(np.asarray(term, dtype=np.float64))
    return act(z, kind), z, s


def _by_group(x, groups):
    """[n, hw, c] -> [n, groups, hw * c / groups]."""
    n, hw, c = x.shape
    return x.reshape(n, hw, groups, c // groups).transpose(0, 2, 1, 3).reshape(n, groups, -1)


def spread(v, c):
    """[n, groups] -> [n, 1, c]."""
    return np.repeat(v, c // v.shape[1], axis=1)[:, None, :]


def group_norm(x, groups, weight, bias, eps):
    """(z, xhat, mean, rstd) of x [n, hw, c] in float64; the activation is act(z)."""
    x = np.asarray(x, dtype=np.float64)
    g = _by_group(x, groups)
    mean = g.mean(-1)
    rstd = 1 / np.sqrt(((g - mean[..., None]) ** 2).mean(-1) + eps)
    xhat = (x - spread(mean, x.shape[2])) * spread(rstd, x.shape[2])
    return xhat * weight + bias, xhat, mean, rstd


def group_norm_backward(dy, x, mean, rstd, groups, weight, bias, kind, z=None):
    """(dx, dweight, dbias, parts) in float64 from given mean and rstd.  z: the values whose activation is
    taken (for a ReLU whose corner is decided in another precision); parts: (xhat, z, dz, d)."""
    c = x.shape[2]
    x, dy, weight, bias = (np.asarray(t, dtype=np.float64) for t in (x, dy, weight, bias))
    xhat = (x - spread(np.asarray(mean, np.float64), c)) * spread(np.asarray(rstd, np.float64), c)
    if z is None:
        z = xhat * weight + bias
    dz = dy * act_grad(np.asarray(z, np.float64), kind)
    d = dz * weight
    m1, m2 = (spread(_by_group(t, groups).mean(-1), c) for t in (d * xhat, d))
    dx = spread(np.asarray(rstd, np.float64), c) * (d - m2 - xhat * m1)
    return dx, (dz * xhat).sum((0, 1)), dz.sum((0, 1)), (xhat, z, dz, d)


def _fp8_table(fmt: int) -> np.ndarray:
    """The values of the 256 codes."""
    bits, bias = (2, 15) if fmt else (3, 7)
    v = np.empty(256)
    for code in range(256):
        e, m = code >> bits & (1 << 7 - bits) - 1, code & (1 << bits) - 1
        if fmt and e == 31:
            x = np.inf if m == 0 else np.nan
        elif not fmt and code & 127 == 127:
            x = np.nan
        else:
            x = m * 2.0 ** (1 - bias - bits) if e == 0 else (1 + m / (1 << bits)) * 2.0 ** (e - bias)
        v[code] = -x if code >= 128 else x
    return v


FP8 = [_fp8_table(0), _fp8_table(1)]
FP8_MOST = [448.0, 57344.0]


def _fp8_nearest(a: np.ndarray, fmt: int) -> np.ndarray:
    """Codes without a sign of magnitudes a >= 0 up to the format's largest value: the nearest, halves to even."""
    top = 0x7e if fmt == 0 else 0x7b
    levels = FP8[fmt][:top + 1]
    low = np.clip(np.searchsorted(levels, a, side="right") - 1, 0, top)
    high = np.minimum(low + 1, top)
    below, above = a - levels[low], levels[high] - a
    return np.where((above < below) | ((above == below) & (low % 2 == 1)), high, low).astype(np.uint8)


def fp8_quantize(x: np.ndarray, fmt: int = 0):
    """Codes and scales of x [rows, k] (any float type; exact in float64)."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    k1 = (k + 127) // 128
    b = np.zeros((rows, k1 * 128))
    b[:, :k] = x
    b = b.reshape(rows, k1, 128)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    s = np.zeros((rows, k1), dtype=np.int64)
    # the smallest byte under which the block fits: raised from one that is too small
    s[top > 0] = np.frexp(top[top > 0])[1] - 1 - (15 if fmt else 8) + 127 - 1
    s = np.maximum(s, 0)
    while True:
        small = top > FP8_MOST[fmt] * np.ldexp(1.0, s - 127)
        if not small.any():
            break
        s = s + small
    codes = _fp8_nearest(np.ldexp(np.abs(b), (127 - s)[..., None]), fmt) + 128 * np.signbit(b).astype(np.uint8)
    codes[bad] = 0
    s[bad] = 255
    scales = np.zeros((rows, (k1 + 3) // 4 * 4), dtype=np.uint8)
    scales[:, :k1] = s
    return (np.ascontiguousarray(codes.transpose(1, 0, 2)),
            np.ascontiguousarray(scales.reshape(rows, -1, 4).transpose(1, 0, 2)))


def fp8_values(codes: np.ndarray, scales: np.ndarray, k: int, fmt: int = 0) -> np.ndarray:
    """float64 [rows, k]: the values that codes and scales stand for."""
    k1, rows, _ = codes.shape
    s = scales.astype(np.int64).transpose(1, 0, 2).reshape(rows, -1)[:, :k1]
    v = np.ldexp(FP8[fmt][codes.transpose(1, 0, 2)], (s - 127)[..., None])
    v[s == 255] = np.nan
    return v.reshape(rows, k1 * 128)[:, :k]


def fp8_matmul(a, w, k: int, fmt: int = 0, bias=None, residual=None, kind: int = 0):
    """(y, z, s): the product after the activation, before it, and the sum of its terms' magnitudes."""
    av, wv = fp8_values(*a, k, fmt), fp8_values(*w, k)
    z, s = av @ wv.T, np.abs(av) @ np.abs(wv).T
    for term in (bias, residual):
        if term is not None:
            z, s = z + np.asarray(term, dtype=np.float64), s + np.abs(np.asarray(term, dtype=np.float64))
    return act(z, kind), z, s


def gated(x, gate, up, k: int, kind: int):
    """(y, g, u, sg, su): act(g) u, both projections and the sums of their terms' magnitudes."""
    xv, gv, uv = (fp8_values(*t, k) for t in (x, gate, up))
    g, u = xv @ gv.T, xv @ uv.T
    return act(g, kind) * u, g, u, np.abs(xv) @ np.abs(gv).T, np.abs(xv) @ np.abs(uv).T


def gated_backward(dy, g, u, kind: int):
    """(dgate, dup) from the projections."""
    return dy * u * act_grad(g, kind), dy * act(g, kind)


def rms_norm(h, weight, eps):
    """(y, rstd) of h [rows, c] in float64."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * (1.0 if weight is None else np.asarray(weight, np.float64)), rstd


def rms_norm_backward(dy, h, rstd, weight, dh=None):
    """(dx, dweight) in float64 from a given rstd."""
    dy, h, rstd = (np.asarray(t, dtype=np.float64) for t in (dy, h, rstd))
    xhat = h * rstd[:, None]
    d = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd[:, None] * (d - xhat * (d * xhat).mean(-1, keepdims=True))
    return dx if dh is None else dx + np.asarray(dh, np.float64), (dy * xhat).sum(0)
