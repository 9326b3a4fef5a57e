"""MXFP4 and its products from their definitions, in numpy float64 (no library code): E2M1
values by their bit fields, rounding by comparing distances to all eight magnitudes, products
summed exactly enough in float64 (every product is a small multiple of a power of two)."""
import math

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0 if c == 0 else (0.5 * (c & 1) if c < 2 else (1 + 0.5 * (c & 1)) * 2.0 ** ((c >> 1) - 1))
                       for c in range(8)])


def blocks(k):
    return -(-k // BLOCK)


def quant(x):
    """(codes (R, 16 KB) uint8, scale (R, KB) uint8) of a 2-D float16 array along its rows."""
    R, K = x.shape
    kb = blocks(K)
    v = np.zeros((R, kb * BLOCK))
    v[:, :K] = x.astype(np.float64)
    v = v.reshape(R, kb, BLOCK)
    bad = ~np.isfinite(v).all(-1)
    amax = np.where(np.isfinite(v), np.abs(v), 0.0).max(-1)
    e = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1.0))[1] - 3, 0)
    e = np.where(bad, 0, e)
    u = np.where(np.isfinite(v), v, 0.0) * 2.0 ** -e[..., None]
    dist = np.abs(np.abs(u)[..., None] - MAGNITUDES)
    best = dist.min(-1, keepdims=True)
    code = np.zeros(u.shape, dtype=np.uint8)
    for c in list(range(1, 8, 2)) + list(range(0, 8, 2)):  # even codes last: they win ties
        code = np.where(dist[..., c] == best[..., 0], np.uint8(c), code)
    code = code | (np.signbit(v).astype(np.uint8) << 3)
    code[bad] = 0
    code = code.reshape(R, kb * BLOCK)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scale


def values(codes, scale):
    """float64 (R, 32 KB) of an MXFP4 matrix."""
    R, kb = scale.shape
    c = np.empty((R, codes.shape[1] * 2), dtype=np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return (v.reshape(R, kb, BLOCK) * s[..., None]).reshape(R, kb * BLOCK)


def to_half(x):
    with np.errstate(over="ignore"):
        return x.astype(np.float16)


def random_matrix(rng, R, K, lo=118, hi=132):
    """Random codes (zero past K) and scales with exponents lo .. hi."""
    kb = blocks(K)
    code = rng.integers(0, 16, (R, kb * BLOCK), dtype=np.uint8)
    code[:, K:] = 0
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), rng.integers(lo, hi + 1, (R, kb), dtype=np.uint8)


def product(A, B, relu=False):
    """(A B^T, bound) in float64: the bound is half a binary16 step of the result (2^-11 of it,
    2^-25 where it is subnormal), and for each of the K additions one float32 step (2^-23, for
    adders that truncate) of the sum of the magnitudes, which no partial sum exceeds."""
    ref = A @ B.T
    mag = np.abs(A) @ np.abs(B).T
    tol = np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + A.shape[1] * 2.0 ** -23 * mag
    if relu:
        ref = np.where(ref > 0, ref, 0.0)
    return ref, tol


def check(c, ref, tol, what=""):
    """c float16 against ref within tol; NaN where ref is NaN, infinite where binary16 has no
    larger value (ref past 65520, half a step over the largest)."""
    c = c.astype(np.float64)
    nan = np.isnan(ref)
    assert (np.isnan(c) == nan).all(), f"{what}: NaN in the wrong places"
    over = np.abs(ref) >= 65520 * (1 + 2.0 ** -9)
    near = (np.abs(ref) >= 65520 * (1 - 2.0 ** -9)) & ~over
    assert (np.isinf(c[over])).all() and (np.sign(c[over]) == np.sign(ref[over])).all(), what
    ok = ~nan & ~over & ~near
    err = np.abs(c[ok] - ref[ok])
    worst = float((err / tol[ok]).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} of the tolerance"
    return worst


def sqrt_k(k):
    return math.sqrt(max(k, 1))
