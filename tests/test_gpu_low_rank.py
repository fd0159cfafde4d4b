"""The orthogonalised update of matrices of few directions, through the library: the gradients of few
tokens or of few live channels have no more, and roundings in the directions that they lack grow."""
import numpy as np
import pytest
import torch

from oracle import layers
from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def off(got, want):
    return np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)


# one launch, the tiled form with a side of 64, long and tall, and rows beyond 512 columns
@pytest.mark.parametrize("rows,cols", [(30, 40), (64, 147), (147, 64), (40, 500), (40, 600), (65, 147), (257, 300), (300, 257), (700, 800)])
@pytest.mark.parametrize("kind", layers.LOW_RANK)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_directions(rows, cols, kind, dtype):
    """A bf16 is at most 2^-8 off; the products' roundings, by the oracle's at the same places, at most as
    much.  (A bf16 input is rounded first, which gives it more directions than it was made with.)"""
    say("low rank", rows, cols, kind, dtype)
    g = [torch.from_numpy(layers.low_rank(rows, cols, kind, seed)).to(dtype) for seed in range(3)]
    got = gq().orthogonalise(torch.stack(g).cuda())
    for i in range(3):
        d = off(got[i], layers.orthogonalise(g[i].double().numpy()))
        assert d <= 2.0 ** -7, (i, d)


@pytest.mark.parametrize("rows,cols", [(64, 147), (40, 600), (300, 257), (700, 800)])
@pytest.mark.parametrize("kind", layers.LOW_RANK)
@pytest.mark.parametrize("steps", [2, 3, 8])
def test_more_steps_and_fewer(rows, cols, kind, steps):
    """As above, and what fp32 itself leaves in directions that the matrix lacks: a few 2^-24 a step, each
    grown at most 3.45^7-fold, below 2^-10 of the norm a step, 2^-7 in all."""
    say("low rank, steps", rows, cols, kind, steps)
    g = layers.low_rank(rows, cols, kind, 5)
    d = off(gq().orthogonalise(torch.from_numpy(g).cuda(), steps=steps), layers.orthogonalise(g, steps))
    assert d <= 2.0 ** -7 + (2.0 ** -7 if steps > 5 else 0.0), d


@pytest.mark.parametrize("rows,cols", [(2, 2), (9, 33), (64, 64), (64, 512), (130, 130), (512, 300)])
def test_all_elements_alike(rows, cols):
    """Every rounding has the same sign: at most 2^-6 by the oracle's."""
    say("elements alike", rows, cols)
    g = torch.full((rows, cols), 0.37)
    d = off(gq().orthogonalise(g.cuda()), layers.orthogonalise(g.double().numpy()))
    assert d <= 2.0 ** -6, d


@pytest.mark.parametrize("side", [1100, 2000])
def test_one_direction_in_few_rows_of_a_large_matrix(side):
    say("few rows of a large matrix", side)
    g = np.zeros((side, 2100), np.float32)
    rng = np.random.default_rng(side)
    g[[5, side // 2, side - 1]] = np.outer([0.5, -0.7, 0.4], rng.standard_normal(2100))
    want = layers.orthogonalise(g[[5, side // 2, side - 1]])      # the other rows stay zero
    got = gq().orthogonalise(torch.from_numpy(g).cuda())
    assert off(got[[5, side // 2, side - 1]], want) <= 2.0 ** -7
    assert got.double().norm().item() <= np.linalg.norm(want) * (1 + 2.0 ** -7)


def test_coefficients_that_roundings_escape():
    """Refused, where finite numbers would come out as NaN after some steps."""
    say("coefficients refused")
    g = gq()
    x = torch.ones(64, 147, device="cuda")
    for coefficients, steps in (((5.0, -20.0, 16.0), 5), ((3.0, -4.0, 0.0), 32), ((50.0, -49.0, 1e-18), 1)):
        with pytest.raises(g.GQError):
            g.orthogonalise(x, steps=steps, coefficients=coefficients)
    assert torch.isfinite(g.orthogonalise(x, steps=32)).all()
