"""Pins of the MXFP4 reference used by the GPU tests (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

import mx_reference as mx


def test_magnitudes():
    assert mx.MAGNITUDES.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def test_ties_go_to_the_even_code():
    # amax 4 -> scale 1; every midpoint of the grid, and the values past 6 a block can hold
    x = np.zeros((1, 32), dtype=np.float16)
    x[0, :9] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.25, -3.5]
    q, s = mx.quant(x)
    assert s[0, 0] == 127
    assert mx.values(q, s)[0, :9].tolist() == [4, 0, 1, 1, 2, 2, 4, 0, -4]
    x[0, 0] = 7.9  # still scale 1: saturates at 6; 5 is a tie between 4 and 6
    x[0, 1] = 5
    q, s = mx.quant(x)
    assert s[0, 0] == 127 and mx.values(q, s)[0, :2].tolist() == [6, 4]


@pytest.mark.parametrize("amax,e", [(2.0 ** -24, -26), (6.0, 0), (65504.0, 13), (0.0, 0), (1.0, -2)])
def test_scales(amax, e):
    x = np.zeros((1, 40), dtype=np.float16)
    x[0, 5] = amax
    q, s = mx.quant(x)
    assert s[0].tolist() == [e + 127, 127]
    assert q[0, 16:].tolist() == [0] * 16


def test_nonfinite_blocks():
    x = np.ones((2, 64), dtype=np.float16)
    x[0, 3], x[1, 40] = np.inf, np.nan
    q, s = mx.quant(x)
    assert s.tolist() == [[255, 125], [125, 255]]
    assert (q[0, :16] == 0).all() and (q[1, 16:] == 0).all()


def test_nearest_by_exact_arithmetic():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((4, 50)) * 2.0 ** rng.integers(-20, 12, (4, 1))).astype(np.float16)
    q, s = mx.quant(x)
    v = mx.values(q, s)
    for i in range(4):
        for j in range(50):
            scale = Fraction(2) ** (int(s[i, j // 32]) - 127)
            got = abs(Fraction(float(v[i, j])) - Fraction(float(x[i, j])))
            best = min(abs(Fraction(float(m)) * sg * scale - Fraction(float(x[i, j]))) for m in mx.MAGNITUDES for sg in (1, -1))
            assert got == best


def test_product_bound_catches_a_wrong_scale():
    rng = np.random.default_rng(4)
    A, sa = mx.random_matrix(rng, 16, 256)
    B, sb = mx.random_matrix(rng, 16, 256)
    ref, tol = mx.product(mx.values(A, sa), mx.values(B, sb))
    sa[:, 2] += 1
    wrong, _ = mx.product(mx.values(A, sa), mx.values(B, sb))
    assert (np.abs(wrong - ref) > tol).mean() > 0.5
