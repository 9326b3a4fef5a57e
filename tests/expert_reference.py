"""Definitions of the expert layer's operators in numpy (no library code): sorting, rows out and back,
the products and their gradients, in float64 where numbers are computed."""
import numpy as np

HALF16 = 2.0 ** -11
TINY16 = 2.0 ** -25


def sort(ids, experts):
    """(offsets, order, place) of the slots of ids (T, k)."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    perm = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[perm], np.arange(experts + 1)).astype(np.int32)
    order = np.full(flat.size, -1, dtype=np.int32)
    order[: offsets[-1]] = perm[: offsets[-1]]
    place = np.full(flat.size, -1, dtype=np.int32)
    place[order[: offsets[-1]]] = np.arange(offsets[-1])
    return offsets, order, place.reshape(ids.shape)


def gather(x, place, out):
    """out with x[t] at every place of token t."""
    out = out.copy()
    for t, j in zip(*np.nonzero(place >= 0)):
        out[place[t, j]] = x[t]
    return out


def slots(y, place):
    """y's row of every slot (T, k, H) float64, zeros for none."""
    got = y.astype(np.float64)[np.maximum(place, 0)]
    got[place < 0] = 0.0
    return got


def combine(y, place, weights):
    """(sums, sums of magnitudes) (T, H)."""
    rows = slots(y, place)
    w = np.ones(place.shape) if weights is None else weights.astype(np.float64)
    rows = np.where((place >= 0)[..., None], rows * w[..., None], 0.0)
    return rows.sum(1), np.abs(rows).sum(1)


def clamped(offsets, rows):
    o = np.clip(np.asarray(offsets, dtype=np.int64), 0, rows)
    return [(int(a), int(max(a, b))) for a, b in zip(o[:-1], o[1:])]


def products(a, b, offsets, trans_b, out):
    """out (float64) with a[p] @ op(b[e]) in the rows of every expert, and the sums of magnitudes."""
    out, size = out.astype(np.float64), np.zeros(out.shape)
    for e, (lo, hi) in enumerate(clamped(offsets, len(a))):
        w = b[e].astype(np.float64)
        w = w.T if trans_b else w
        x = a[lo:hi].astype(np.float64)
        out[lo:hi], size[lo:hi] = x @ w, np.abs(x) @ np.abs(w)
    return out, size


def products_tn(a, b, offsets):
    got = [a[lo:hi].astype(np.float64).T @ b[lo:hi].astype(np.float64) for lo, hi in clamped(offsets, len(a))]
    return np.stack(got)


def product_bound(want, size, terms):
    """Half a step of the result and a float32 rounding of every term's partial sum (2^-23 of the sum of
    magnitudes for each of `terms` additions covers any order of them)."""
    return np.abs(want) * HALF16 + TINY16 + terms * 2.0 ** -23 * size


def to_half(x):
    """float64 to binary16, to nearest even (numpy rounds float64 directly)."""
    with np.errstate(over="ignore"):
        return x.astype(np.float16)
