"""Which coefficients the orthogonalised update takes: the library's own rule, compiled for the host (CPU
only)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "allreduce_compatible_gradient_amd", "csrc")
SHIM = """
#include "gq_range.h"
extern "C" int stays(int32_t steps, double a, double b, double c) { return gq::ortho_stays(steps, a, b, c); }
"""


@pytest.fixture(scope="module")
def stays(tmp_path_factory):
    d = tmp_path_factory.mktemp("range")
    (d / "shim.cpp").write_text(SHIM)
    lib = str(d / "shim.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, str(d / "shim.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).stays
    f.argtypes = [ctypes.c_int32] + [ctypes.c_double] * 3
    return f


# with convergence to 1 (the last two), and sets in use that overshoot it
TAKEN = [layers.QUINTIC, (4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037),
         (2.8769, -3.1427, 1.2046), (2.8366, -3.0525, 1.2012), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0), (2.0, -1.5, 0.5),
         (1.0, 0.0, 0.0), (0.0, 0.0, 0.0)]


@pytest.mark.parametrize("coefficients", TAKEN)
@pytest.mark.parametrize("steps", [1, 5, 32])
def test_taken(stays, coefficients, steps):
    assert stays(steps, *coefficients)


@pytest.mark.parametrize("c", [0.0, 1e-18, -1e-18, 1e-30, 5e-324, 1e-9])
def test_a_largest_value_between_the_ends(stays, c):
    """p(x) = 50 x - 49 x^3 is 1 at 1 and 19 at 0.58, with next to nothing of the fifth power too, where
    the roots of p' are far apart."""
    assert not stays(1, 50.0, -49.0, c)


def test_against_a_fine_grid(stays):
    """One step is taken exactly where |p| and |b s + c s^2| stay below their bounds on [0, 1]."""
    rng = np.random.default_rng(1)
    x = np.linspace(0, 1, 20001)
    seen = [0, 0]
    for _ in range(2000):
        a, b, c = rng.standard_normal(3) * 10.0 ** rng.uniform(-1, 2, 3)
        p, q = np.abs(x * (a + x * x * (b + x * x * c))).max(), np.abs(x * (b + x * c)).max()
        if 0.9 < p / 7.5 < 1.1 or 0.9 < q / 60.0 < 1.1:     # near a bound, which roundings may move
            continue
        assert stays(1, a, b, c) == (p < 7.5 and q < 60.0), (a, b, c, p, q)
        seen[int(p < 7.5 and q < 60.0)] += 1
    assert min(seen) > 100


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e308])
def test_not_numbers(stays, bad):
    for i in range(3):
        k = [1.0, 0.0, 0.0]
        k[i] = bad
        assert not stays(1, *k)


# on [0, 1] these stay within [-1, 1], but a rounding past 1 is taken out of it, 9 or 25 times as far a step
ESCAPE = [((5.0, -20.0, 16.0), 5), ((5.0, -20.0, 16.0), 10), ((3.0, -4.0, 0.0), 32), ((-3.0, 4.0, 0.0), 32),
          ((-5.0, 20.0, -16.0), 32)]


@pytest.mark.parametrize("coefficients,steps", ESCAPE)
def test_roundings_that_escape(stays, coefficients, steps):
    assert not stays(steps, *coefficients)


def test_what_is_taken_stays_finite(stays):
    """Coefficients near the rule's border, on matrices of one direction, of equal elements and of a broad
    spectrum, with the products' roundings: the values that halves hold are never left."""
    rng = np.random.default_rng(3)
    matrices = [layers.low_rank(64, 147, "rank1", 1), layers.low_rank(70, 90, "rows", 2), np.full((40, 60), 0.37),
                rng.standard_normal((30, 40)), np.eye(7, 9)]
    taken = escaped = 0
    while taken < 150:
        # maps of [0, 1] to about itself: any a and c, b so that p(1) lies within [-1.2, 1.2]
        a, c = rng.uniform(-6, 6), rng.uniform(-16, 16)
        b, steps = rng.uniform(-1.2, 1.2) - a - c, int(rng.integers(4, 33))
        if not stays(steps, a, b, c):
            escaped += 1
            continue
        taken += 1
        for g in matrices:
            with np.errstate(all="ignore"):
                got = layers.orthogonalise_in_halves(g, steps, (a, b, c))
            assert np.all(np.isfinite(got)), (a, b, c, steps)
            assert np.linalg.norm(got, 2) <= 7.5 * (1 + 2.0 ** -7), (a, b, c, steps)
    assert escaped > 50
