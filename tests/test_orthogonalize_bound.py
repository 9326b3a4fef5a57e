"""The bound that the GPU tests of the orthogonalisation use, on the CPU: the kernels' arithmetic,
emulated, is inside it, and arithmetic with fewer bits is not."""
import numpy as np
import pytest

import ns_reference as ns

SHAPES = [(64, 64), (64, 500), (130, 200), (256, 256)]
FEWER = {"high halves alone in the products": dict(gram=False, square=False, apply=False, split_p=False),
         "high halves alone in the square": dict(square=False),
         "A and P in one half": dict(split_p=False),
         "A and P in one half, diagonals inside": dict(split_p=False, diagonals=False),
         "the iterate in one half": dict(split_x=False),
         "everything in one half": dict(split_x=False, split_p=False, diagonals=False)}


@pytest.fixture(scope="module")
def solved():
    out = []
    for shape in SHAPES:
        for name, make in ns.INPUTS.items():
            for steps in (4, 5, 6, 10):
                g = make(np.random.default_rng(sum(shape)), *shape).astype(np.float32)
                ref = ns.iterates(g, steps)[-1]
                out.append((f"{name} {shape} {steps} steps", g, steps, ref, ns.bound(g, ref, steps)))
    return out


def test_the_kernels_arithmetic_is_inside(solved):
    for what, g, steps, ref, bound in solved:
        assert np.linalg.norm(ns.rounded(ns.emulate(g, steps)) - ref) <= bound, what


@pytest.mark.parametrize("name", FEWER)
def test_fewer_bits_are_not(solved, name):
    """On random matrices always (the square's low halves where m is no small part of n); under
    one dominant direction the result hangs on the low half of the iterate."""
    for what, g, steps, ref, bound in solved:
        err = np.linalg.norm(ns.rounded(ns.emulate(g, steps, **FEWER[name])) - ref)
        if what.startswith("dominated"):
            seen = "iterate" in name or "products" in name
        else:
            seen = "square" not in name or g.shape[1] < 2 * g.shape[0]
        assert err > bound or not seen, what
