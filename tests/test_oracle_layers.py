"""The definitions of 8-bit rows, embeddings and the orthogonalised update against closed forms and
differences (CPU only)."""
import numpy as np
import pytest

from oracle import layers, lm


def test_codes_of_known_rows():
    x = np.array([[127, -63.5, 0.5, 1.5, -0.0], [0, 0, 0, 0, 0], [1e-38, 0, 0, 0, 0], [1, np.nan, 0, 0, 0],
                  [np.inf, 0, 0, 0, 0], [-2, 1, 0, 0, 0]], np.float32)
    codes, scales = layers.quantize(x, layers.NEAREST)
    assert codes.shape == (6, 128) and not codes[:, 5:].any()
    assert codes[0, :5].tolist() == [127, -64, 0, 2, 0] and scales[0] == 1.0
    assert not codes[1:5].any() and scales[1] == 0 and scales[2] == 0 and np.isnan(scales[3]) and np.isnan(scales[4])
    assert codes[5, :2].tolist() == [-127, 64] and scales[5] == np.float32(2) / np.float32(127)


def test_nearest_is_within_half_a_code():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((20, 300)).astype(np.float32) * np.exp2(rng.integers(-40, 40, (20, 1))).astype(np.float32)
    codes, scales = layers.quantize(x, layers.NEAREST)
    v = codes[:, :300] * scales[:, None].astype(np.float64)
    # half a code, and the roundings of scale and inv (2^-24 of the value each)
    assert np.all(np.abs(v - x) <= scales[:, None].astype(np.float64) * 0.5 + np.abs(x) * 2.0 ** -22)
    assert np.all(np.abs(codes).max(1) == 127)


def test_stochastic_is_unbiased():
    x = np.repeat(np.array([[1.0, 0.3, -0.77, 0.004]], np.float32), 4000, 0)
    r = lm.draws(*x.shape, seed=11)
    codes, scales = layers.quantize(x, layers.STOCHASTIC, r)
    mean = (codes[:, :4] * scales[:, None].astype(np.float64)).mean(0)
    # a code's standard deviation is at most half a step: five of them over 4000 draws
    assert np.all(np.abs(mean - x[0]) <= 5 * 0.5 * scales[0] / np.sqrt(4000) + 1e-6)


def test_product_is_of_the_values():
    rng = np.random.default_rng(2)
    a, sa = layers.quantize(rng.standard_normal((3, 40)).astype(np.float32), layers.NEAREST)
    b, sb = layers.quantize(rng.standard_normal((5, 40)).astype(np.float32), layers.NEAREST)
    bias = rng.standard_normal(5)
    want = (a * sa[:, None].astype(np.float64)) @ (b * sb[:, None].astype(np.float64)).T + bias
    assert np.allclose(layers.matmul(a, sa, b, sb, bias)[0], want, rtol=1e-12, atol=1e-12)


def test_embedding_gradient_by_differences():
    rng = np.random.default_rng(3)
    table, ids = rng.standard_normal((6, 4)), np.array([2, -1, 2, 5, 6, 0, 2])
    w = rng.standard_normal((7, 4))
    grad, mass, count = layers.embedding_grad(w, ids, 6, 1.5)
    for v in range(6):
        for e in range(4):
            d = np.zeros_like(table)
            d[v, e] = 1e-3
            diff = ((layers.embedding(table + d, ids, 1.5) - layers.embedding(table - d, ids, 1.5)) * w).sum() / 2e-3
            assert abs(diff - grad[v, e]) < 1e-9
    assert count.tolist() == [1, 0, 3, 0, 0, 1] and np.all(np.abs(grad) <= mass + 1e-15)


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6), (1, 7), (7, 1)])
def test_orthogonalised_singular_values(shape):
    g = np.random.default_rng(4).standard_normal(shape)
    u, s, v = np.linalg.svd(g, full_matrices=False)
    a, b, c = layers.QUINTIC
    s = s / np.sqrt((s * s).sum())
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(layers.orthogonalise(g), (u * s) @ v, atol=1e-10)
    assert not layers.orthogonalise(np.zeros(shape)).any()


def test_roundings_stay_small():
    """The library's roundings on matrices of a side of 48: at most 2^-8 off, a bf16's half step, 2^-9 in
    the root mean square, the largest part of it."""
    rng = np.random.default_rng(5)
    for g in (rng.standard_normal((48, 80)), rng.standard_normal((80, 48)) ** 3,
              rng.standard_normal((48, 4)) @ rng.standard_normal((4, 48)) + 0.05 * rng.standard_normal((48, 48))):
        want, got = layers.orthogonalise(g), layers.orthogonalise_rounded(g)
        assert np.linalg.norm(got - want) <= 2.0 ** -8 * np.linalg.norm(want)
