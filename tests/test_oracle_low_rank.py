"""The orthogonalised update of matrices of few directions: how far the library's roundings take it, and
what keeps them small (CPU only)."""
import numpy as np
import pytest

from oracle import layers

# a bf16 is at most 2^-8 off, and what the products' roundings leave at most as much
BOUND = 2.0 ** -7


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("kind", layers.LOW_RANK)
@pytest.mark.parametrize("rows,cols", [(40, 500), (64, 147), (147, 64), (65, 147), (257, 300), (300, 257)])
def test_few_directions(rows, cols, kind):
    for seed in range(3):
        g = layers.low_rank(rows, cols, kind, seed)
        assert off(layers.orthogonalise_in_halves(g), layers.orthogonalise(g)) <= BOUND, seed


@pytest.mark.parametrize("kind", layers.LOW_RANK)
@pytest.mark.parametrize("rows,cols", [(64, 147), (257, 300)])
def test_eight_steps(rows, cols, kind):
    g = layers.low_rank(rows, cols, kind, 1)
    assert off(layers.orthogonalise_in_halves(g, 8), layers.orthogonalise(g, 8)) <= BOUND


def test_what_the_diagonal_apart_would_leave():
    """One direction in two rows of 300: with the diagonal on X itself and the rest on its halves, the
    roundings that only one of them has grow 3.4-fold a step, to more than 1%."""
    g = np.zeros((300, 400), np.float32)
    g[:2] = np.outer([0.8, 0.6], np.random.default_rng(1).standard_normal(400))
    want = layers.orthogonalise(g)
    assert off(layers.orthogonalise_rounded(g), want) > 1e-2
    assert off(layers.orthogonalise_in_halves(g), want) <= BOUND


def test_all_elements_alike():
    """Every rounding has the same sign then: sizes 2 to 500 are at most 2^-6 off."""
    rng = np.random.default_rng(2)
    for _ in range(40):
        rows, cols = (int(np.exp(rng.uniform(np.log(2), np.log(500)))) for _ in range(2))
        g = np.full((rows, cols), 0.37)
        assert off(layers.orthogonalise_in_halves(g), layers.orthogonalise(g)) <= 2.0 ** -6, (rows, cols)


@pytest.mark.parametrize("shape", [(20, 21), (64, 147), (100, 130), (300, 257)])
def test_a_broad_spectrum_is_as_near_as_before(shape):
    """Half as far again as with the diagonal apart in every step, at most."""
    for seed in range(3):
        g = np.random.default_rng(seed).standard_normal(shape)
        want = layers.orthogonalise(g)
        assert off(layers.orthogonalise_in_halves(g), want) <= 1.5 * off(layers.orthogonalise_rounded(g), want)
