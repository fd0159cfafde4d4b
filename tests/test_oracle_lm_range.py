"""The 64-bit definition of the distillation loss where plain probabilities leave the range of
numbers, against hand-worked values and difference quotients (CPU only)."""
import numpy as np
import pytest

from oracle import lm


@pytest.mark.parametrize("gap", [30.0, 100.0, 1000.0])
def test_distill_bucket_far_below(gap):
    """The rest `gap` below two taught entries: log q_R = -gap + log 3 - log 2, its mass spread as the
    rest's own softmax, and the gradient is the difference quotient."""
    z = np.array([[gap, gap, 0.0, 0.0, 0.0]])
    ids, p = np.array([[0, 1]]), np.array([[0.5, 0.25]])
    loss, grad, _ = lm.distill(z, ids, np.log(p), 1.0, True)
    want = 0.5 * np.log(0.5 / 0.5) + 0.25 * np.log(0.25 / 0.5) + 0.25 * (np.log(0.25) + gap - np.log(1.5))
    assert abs(loss[0] - want) < 1e-9 * (1 + gap)
    assert np.allclose(grad[0], [0.0, 0.25, -0.25 / 3, -0.25 / 3, -0.25 / 3], atol=1e-9)
    h = 1e-4
    for v in range(5):
        up, down = z.copy(), z.copy()
        up[0, v] += h
        down[0, v] -= h
        d = (lm.distill(up, ids, np.log(p), 1.0, True)[0] - lm.distill(down, ids, np.log(p), 1.0, True)[0]) / (2 * h)
        assert abs(d[0] - grad[0, v]) < 1e-6


@pytest.mark.parametrize("level", [-2000.0, -100.0, 100.0, 2000.0])
def test_distill_without_a_tail_knows_proportions_only(level):
    rng = np.random.default_rng(5)
    z, lps = rng.normal(size=(1, 8)), np.log([[0.5, 0.3, 0.2]])
    ids = np.array([[4, 0, 6]])
    want, got = (lm.distill(z, ids, lps + c, 1.5, False) for c in (0.0, level))
    assert np.allclose(got[0], want[0], rtol=1e-10) and np.allclose(got[1], want[1], atol=1e-10)


@pytest.mark.parametrize("vocab,total", [(12, 0.4), (12, 1.5), (5, 0.4), (5, 1.0), (5, 1.5)])
def test_distill_gradient_with_any_mass(vocab, total):
    """Entries that sum to less or more than one, with a rest and (5 of 5 taught) without."""
    rng = np.random.default_rng(6)
    z, p = rng.normal(size=(1, vocab)), rng.random((1, 5)) + 0.1
    ids, lps = np.arange(5)[None], np.log(total * p / p.sum())
    _, grad, _ = lm.distill(z, ids, lps, 1.5, True)
    h = 1e-5
    for v in range(vocab):
        up, down = z.copy(), z.copy()
        up[0, v] += h
        down[0, v] -= h
        d = (lm.distill(up, ids, lps, 1.5, True)[0] - lm.distill(down, ids, lps, 1.5, True)[0]) / (2 * h)
        assert abs(d[0] - grad[0, v]) < 1e-8
