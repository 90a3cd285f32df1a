"""Microscaled 4-bit floating point, the products and the norms around a block,
from their definitions in 64 bits on the CPU (numpy)."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x [rows][cols] -> (codes 0..15 [rows][cols], scale bytes [rows][cols/32])."""
    v = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    with np.errstate(invalid="ignore"):
        top = np.abs(v).max(-1)
    bad = ~np.isfinite(v).all(-1)
    safe = np.where(bad | (top == 0), 1.0, top)
    e = np.clip(np.frexp(safe)[1] - 1 - 2, -127, 127)
    byte = np.where(bad, 255, np.where(top == 0, 0, e + 127)).astype(np.uint8)
    q = np.abs(np.where(bad[..., None], 0.0, v)) / np.exp2(e)[..., None]
    dist = np.abs(np.minimum(q, 6.0)[..., None] - MAGNITUDES)
    # nearest; of two equally near ones the even code
    code = np.argmin(dist + np.array([0.0, 1e-9] * 4) * (dist == dist.min(-1, keepdims=True)), -1)
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(v))
    return code.reshape(x.shape).astype(np.uint8), byte


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def values(codes, byte):
    """codes 0..15 [..., cols], byte [..., cols/32] -> values in 64 bits."""
    v = np.where(codes >= 8, -1.0, 1.0) * MAGNITUDES[codes & 7]
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return (v.reshape(*byte.shape, 32) * s[..., None]).reshape(codes.shape)


def rounding(dtype_eps, smallest, v):
    """Half a step of a type at v."""
    return np.abs(v) * dtype_eps / 2 + smallest / 2


def product(x, w, swiglu):
    """x [rows][cols], w [n][cols] in 64 bits -> (out, tolerance before the
    output's rounding).  The sum over a block of 32 is a multiple of a quarter of
    the two scales below 4608 of them, so it is exact in 24 bits.  The sums over
    the n = cols / 32 blocks, in any order and grouping, are at most n + 4
    additions of 2^-23 (24 bits, nearest or cut) of the absolute terms.
    swiglu: |silu'| < 1.1 and |silu(v)| <= |v|; the exponential, the sum, the
    reciprocal and the products are 12 roundings of 2^-23 at most; below v = -87,
    where the exponential overflows, the result is below 87 e^-87 |u| < 2^-118 |u|."""
    y = x @ w.T
    d = (x.shape[1] / 32 + 4) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    if not swiglu:
        return y, d
    n = w.shape[0] // 2
    g, u, dg, du = y[:, :n], y[:, n:], d[:, :n], d[:, n:]
    with np.errstate(over="ignore"):
        silu = g / (1.0 + np.exp(-g))
    out = silu * u
    tol = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du
    return out, tol + 12 * 2.0 ** -23 * np.abs(out) + 2.0 ** -118 * np.abs(u)


def norm(v, weight, offset, eps):
    u = 1.0 if weight is None else offset + weight.astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * u
