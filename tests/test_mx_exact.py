"""What the bit-for-bit product tests see along a long K, on the CPU: one code or one scale that is
wrong changes results that the rounding bound lets pass."""
import numpy as np

import mx_reference as mx


def operands(rng, M, N, K):
    A, sa = mx.random_matrix(rng, M, K, 124, 126)
    B, sb = mx.random_matrix(rng, N, K, 124, 126)
    return A, sa, B, sb


def test_one_dropped_k_shows_in_the_exact_result_only():
    rng = np.random.default_rng(1)
    A, sa, B, sb = operands(rng, 40, 40, 8192)
    a, b = mx.values(A, sa), mx.values(B, sb)
    ref, tol = mx.product(a, b)
    a[:, 5000] = 0.0
    wrong = a @ b.T
    changed = wrong != ref
    assert ((wrong.astype(np.float16) != ref.astype(np.float16))[changed]).mean() > 0.5
    assert (np.abs(wrong.astype(np.float16) - ref) <= tol).mean() > 0.9


def test_one_wrong_scale_shows():
    rng = np.random.default_rng(2)
    A, sa, B, sb = operands(rng, 40, 40, 8192)
    ref = mx.values(A, sa) @ mx.values(B, sb).T
    sb[:, 255] ^= 1
    wrong = mx.values(A, sa) @ mx.values(B, sb).T
    assert (wrong.astype(np.float16) != ref.astype(np.float16)).mean() > 0.9
