"""float64 definition of the root-mean-square norm with the residual's addition, of its E4M3 output
and of its gradient, with the error bounds of float32 sums and one rounding (numpy, no library code).

Where the bounds come from, with u = 2^-24 (a float32 rounding): the sum of squares adds at most 16
values a thread, then at most 6 + 16 partial sums, and every square adds a rounding of its own that
fma avoids: below 40 u; the division by K, eps, the square root, its reciprocal and two products are
6 more, the first 42 halved by the root: y is within 28 u < 2^-19 of its value before the rounding to
binary16 (half a step: 2^-11 of the value, 2^-25 below the normal range)."""
import numpy as np

HALF16 = 2.0 ** -11
TINY16 = 2.0 ** -25
Y_REL = 2.0 ** -19


def stored(x, r):
    """h as it is stored (x and r float16 or float32 arrays)."""
    if r is None:
        return x
    return (x.astype(np.float64) + r.astype(np.float64)).astype(r.dtype)


def norm(h, w, eps):
    """(y, rstd) in float64."""
    h, w = h.astype(np.float64), w.astype(np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def y_bound(y):
    return np.abs(y) * (HALF16 + Y_REL) + TINY16


def e4m3(v):
    """Nearest E4M3 value of float64 v, ties to even, saturated at 448."""
    a = np.abs(v)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.sign(v) * np.minimum(np.round(a / step) * step, 448.0)


def e4m3_value(code):
    """The value of E4M3 codes (uint8)."""
    c = code.astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (f == 7), np.nan, v)
    return np.where(c & 128, -v, v)


def blocks(y):
    """y in blocks of 128 columns, padded with zeros."""
    rows, k = y.shape
    v = np.zeros((rows, -(-k // 128) * 128))
    v[:, :k] = y
    return v.reshape(rows, -1, 128)


def codes_range(y):
    """(scale, lowest, highest code value): the scale amax / 448 (1 for zeros) and the E4M3 values
    between which y / scale may round, y and the scale each within 2^-18 of their value."""
    v = blocks(y)
    top = np.abs(v).max(-1)
    scale = np.where(top < 2.0 ** -100, 1.0, top / 448.0)
    u = np.where(top[..., None] < 2.0 ** -100, 0.0, v / scale[..., None])
    d = np.abs(u) * 2.0 ** -17
    k = y.shape[1]
    return scale, e4m3(u - d).reshape(len(y), -1)[:, :k], e4m3(u + d).reshape(len(y), -1)[:, :k]


def gradient(dy, h, w, eps, dh=None):
    """(dx, its bound before the rounding, dw, sum |dy xhat|). The bound: rstd, xhat, c and the three
    products of dx are float32 (c a sum of K terms, below 40 u of the mean of their magnitudes): each
    within 2^-18 of the magnitudes that enter it."""
    dy, h, w = dy.astype(np.float64), h.astype(np.float64), w.astype(np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    xhat = h * rstd
    p = w * dy
    c = (p * xhat).mean(1, keepdims=True)
    dx = rstd * (p - xhat * c)
    size = rstd * (np.abs(p) + np.abs(xhat) * np.abs(p * xhat).mean(1, keepdims=True))
    if dh is not None:
        dx, size = dx + dh.astype(np.float64), size + np.abs(dh.astype(np.float64))
    return dx, 2.0 ** -18 * size, (dy * xhat).sum(0), np.abs(dy * xhat).sum(0)
