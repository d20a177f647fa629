"""Plain 64-bit reference of the 4-bit and group norm operators (numpy, CPU), written from their
formulas and sharing no code with the library.

A microscaled tensor of `rows` rows and k columns: blocks of 32 columns, codes of 4 bits (magnitudes 0, 0.5,
1, 1.5, 2, 3, 4, 6 and a sign) and a power of two 2^(s - 127) per block; codes [K1, rows, 64] bytes, scales
[K1, rows, 4] bytes, K1 = ceil(k / 128).
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
