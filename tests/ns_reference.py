"""The Newton-Schulz orthogonalisation from its definition in float64, its arithmetic on pairs of
binary16 halves emulated, and the bound that follows for the kernels (numpy, no library code)."""
import numpy as np

A, B, C = 3.4445, -4.7750, 2.0315


def rounded(x):
    with np.errstate(over="ignore"):
        return x.astype(np.float16).astype(np.float64)


def iterates(g, steps=5, coefficients=(A, B, C)):
    """The steps + 1 iterates of one matrix (m <= n: the transpose of a tall one)."""
    a, b, c = coefficients
    x = g.astype(np.float64)
    x = x.T if x.shape[0] > x.shape[1] else x
    xs = [x / (np.sqrt((x * x).sum()) + 1e-7)]
    for _ in range(steps):
        x = xs[-1]
        s = x @ x.T
        xs.append(a * x + (b * s + c * (s @ s)) @ x)
    return xs


def halves(x):
    hi = rounded(x)
    return hi, rounded((x - hi) * 2048.0) / 2048.0


def emulate(g, steps=5, gram=True, square=True, apply=True, split_p=True, split_x=True, diagonals=True):
    """The steps with what is rounded where, in float64: a False leaves out the low halves in the
    Gram product, in the square, in P times X; holds P, or the iterate, in one half; or leaves the
    diagonals of A and P inside the matrices that are rounded."""
    a, b, c = A, B, C
    f32 = lambda v: v.astype(np.float32).astype(np.float64)
    product = lambda u, v, low: f32(u[0] @ v[0] + (u[0] @ v[1] + u[1] @ v[0] if low else 0.0))
    x = f32(iterates(g, 0)[0])
    eye = np.eye(x.shape[0], dtype=bool)
    X = halves(x)
    for _ in range(steps):
        if not split_x:
            X = (X[0], 0.0 * X[1])
        s = product(X, (X[0].T, X[1].T), gram)
        if diagonals:
            D = s.diagonal().copy()
            s[eye] = 0.0
        else:
            D = np.zeros(len(s))
        E = halves(s)
        if not split_p:
            E = (E[0], 0.0 * E[1])
        q = product(E, E, square)
        e = E[0] + E[1]
        p = b * e + c * ((D[:, None] + D[None]) * e + q)
        P = np.full(len(s), a)
        if diagonals:
            P = a + b * D + c * (D * D + q.diagonal())
            p[eye] = 0.0
        P2 = halves(f32(p))
        if not split_p:
            P2 = (P2[0], 0.0 * P2[1])
        X = halves(f32(P[:, None] * (X[0] + X[1]) + product(P2, X, apply)))
    return X[0] + X[1]


def in_float32(g, steps=5, coefficients=(A, B, C)):
    """The steps with float32 matrices and products."""
    a, b, c = (np.float32(v) for v in coefficients)
    x = iterates(g, 0)[0].astype(np.float32)
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.astype(np.float64)


def bound(g, ref, steps=5):
    """Largest Frobenius error of the kernels' result. Their roundings are those of the halves
    (emulated; a value keeps 22 bits, a product drops lo lo) and of float32 sums (as products in float32
    have them). How much of these a later step amplifies depends on the matrix (what the large
    singular values' roundings put into the small ones' directions grows with those), so both are
    taken from the same matrix; both vary with the signs of the roundings, for which twice their
    sum is allowed. The result's rounding to binary16: at most half a step of each value; on 4096
    values or more the rounding of the exact result stands for that of the computed one (other
    values, the same distribution; 10 % added)."""
    noise = 2 * (np.linalg.norm(emulate(g, steps) - ref) + np.linalg.norm(in_float32(g, steps) - ref))
    if ref.size >= 4096:
        return noise + 1.1 * np.linalg.norm(rounded(ref) - ref)
    step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(ref), 2.0 ** -30))), -14)
    return noise + np.linalg.norm(step * 2.0 ** -11)


def gauss(rng, R, C):
    return rng.standard_normal((R, C)) * 0.02


def directions(rng, R, C):
    """A few strong directions over a floor of noise."""
    return rng.standard_normal((R, 8)) @ rng.standard_normal((8, C)) * 1e-3 + rng.standard_normal((R, C)) * 3e-3


def dominated(eps):
    """One direction over noise eps times as large."""
    def make(rng, R, C):
        return rng.standard_normal((R, 1)) @ rng.standard_normal((1, C)) + eps * rng.standard_normal((R, C))
    return make


INPUTS = {"gauss": gauss, "directions": directions, "dominated 1e-2": dominated(1e-2), "dominated 1e-3": dominated(1e-3),
          "dominated 1e-4": dominated(1e-4)}
