"""The 64-bit definitions of the language-model operators against hand-worked values, closed forms
and difference quotients (CPU only)."""
import numpy as np
import pytest

from oracle import lm


def test_nearest_codes_of_a_block():
    # a = 7.9 scales by 1: saturation at 6; ties 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    x = [7.9, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0, -6.0]
    s, c = lm.encode_block(x, lm.NEAREST)
    assert s == 127
    assert c.tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 15]


@pytest.mark.parametrize("a,nearest,stochastic", [(6.0, 127, 127), (6.01, 127, 128), (4.0, 127, 127),
                                                  (3.99, 126, 127), (3.0, 126, 126), (8.0, 128, 128)])
def test_scale_rules(a, nearest, stochastic):
    assert lm.encode_block([a], lm.NEAREST)[0] == nearest
    assert lm.encode_block([a], lm.STOCHASTIC, [0.5])[0] == stochastic


def test_scales_are_clamped_and_bad_blocks_are_nan():
    assert lm.encode_block([1e-45], lm.NEAREST)[0] == 0
    assert lm.encode_block([0.0, -0.0], lm.STOCHASTIC, [0, 0])[0] == 0
    for bad in (np.nan, np.inf, -np.inf):
        s, c = lm.encode_block([1.0, bad], lm.NEAREST)
        assert s == 255 and not c.any()
    codes, scales = lm.quantize(np.array([[1.0, np.nan]]), lm.NEAREST)
    assert np.isnan(lm.decode(codes, scales, 2)).all()


def test_stochastic_rounding_is_unbiased():
    x = np.array([6.0, 0.1, 0.7, 1.3, 2.2, 3.9, 5.1, -0.4])
    r = np.random.default_rng(1).random((20000, x.size))
    mean = np.mean([lm.decode(*[v[None] for v in _packed(x, d)], x.size)[0] for d in r], 0)
    # the spacing is at most 2, so the standard error of a mean is at most 1 / sqrt(20000)
    assert np.all(np.abs(mean - x) < 6 / np.sqrt(20000))


def _packed(x, d):
    s, c = lm.encode_block(x, lm.STOCHASTIC, d)
    nib = np.zeros(256, np.uint8)
    nib[:x.size] = c
    scales = np.zeros(8, np.uint8)
    scales[0] = s
    return nib[0::2] | (nib[1::2] << 4), scales


def test_logprobs_closed_forms():
    z = np.zeros((1, 8))
    lp, h, ids, tops = lm.logprobs(z, [3], 3)
    assert np.allclose([lp[0], h[0]], [-np.log(8), np.log(8)]) and ids.tolist() == [[0, 1, 2]]
    z[0, 1:] = -np.inf
    lp, h, ids, tops = lm.logprobs(z, [0], 2)
    assert lp[0] == 0 and h[0] == 0 and tops.tolist() == [[0, -np.inf]]
    lp, h, _, _ = lm.logprobs(np.full((1, 4), -np.inf), [0], 1)
    assert np.isneginf(lp[0]) and h[0] == 0


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_distill_gradient_is_the_difference_quotient(tail, temperature):
    rng = np.random.default_rng(3)
    z, t = rng.normal(size=(3, 12)), rng.normal(size=(3, 12)) * 2
    lt = lm.log_softmax(t, temperature)
    ids = np.argsort(-lt, 1)[:, :5]
    lps = np.take_along_axis(lt, ids, 1)
    ids[1, 3] = -1                                  # padding
    ids[2, 4] = ids[2, 0]                           # an id that occurs again
    w = np.array([0.7, 1.3, 2.0])
    _, grad, _ = lm.distill(z, ids, lps, temperature, tail, w)
    h = 1e-5
    for i in range(3):
        for v in range(12):
            up, down = z.copy(), z.copy()
            up[i, v] += h
            down[i, v] -= h
            d = (lm.distill(up, ids, lps, temperature, tail)[0][i]
                 - lm.distill(down, ids, lps, temperature, tail)[0][i]) / (2 * h)
            assert abs(grad[i, v] - w[i] * d) < 1e-8        # third derivatives of order 1, times h^2
    # q and p both sum to one, so a row's gradient sums to zero
    assert np.abs(grad.sum(1)).max() < 1e-12


def test_distill_of_the_teacher_itself_is_zero():
    rng = np.random.default_rng(4)
    z = rng.normal(size=(2, 20))
    lp = lm.log_softmax(z, 1.0)
    ids = np.argsort(-lp, 1)[:, :6]
    loss, grad, _ = lm.distill(z, ids, np.take_along_axis(lp, ids, 1), 1.0, True)
    assert np.abs(loss).max() < 1e-12 and np.abs(grad).max() < 1e-12
