"""The orthogonalised update, through the library: as near to the 64-bit definition as the roundings
that it names take it."""
import numpy as np
import pytest
import torch

from oracle import layers
from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def matrix(rows, cols, kind, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols))
    if kind == "heavy":
        x = x ** 3
    elif kind == "few":
        r = min(4, rows, cols)
        x = 0.1 * x + rng.standard_normal((rows, r)) @ rng.standard_normal((r, cols))
    return torch.from_numpy((x * 1e-3).astype(np.float32))


def check(got, g, steps=5, coefficients=layers.QUINTIC, margin=1.5):
    """Against the definition, relative to it in the Frobenius norm.  The library's roundings, made at
    the same places by the oracle, are errors of the same law: theirs, half as much again for their
    chance, and the fp32 sums' own (2^-24 a step of at most 2^10 added numbers and its growth)."""
    x = g.double().cpu().numpy()
    want = layers.orthogonalise(x, steps, coefficients)
    norm = np.linalg.norm(want)
    own = np.linalg.norm(layers.orthogonalise_rounded(x, steps, coefficients) - want)
    off = np.linalg.norm(got.double().cpu().numpy() - want)
    assert off <= margin * own + 2.0 ** -14 * norm, (off / norm, own / norm)


SHAPES = [(1, 5), (7, 1), (2, 2), (16, 16), (33, 50), (64, 64), (64, 147), (65, 63), (128, 128), (129, 257), (257, 129), (200, 1000),
          (1000, 200), (300, 300), (64, 4096), (31, 2000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", ["normal", "heavy", "few"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_matrix(rows, cols, kind, dtype):
    say("orthogonalise", rows, cols, kind, dtype)
    g = matrix(rows, cols, kind, rows * 7 + cols).to(dtype).cuda()
    got = gq().orthogonalise(g)
    assert got.dtype == BF16 and got.shape == g.shape
    # a handful of numbers has no law: the worst of their roundings is some times the usual one
    check(got, g, margin=1.5 if min(rows, cols) >= 16 else 4.0)


@pytest.mark.parametrize("batch,rows,cols", [(3, 20, 30), (43, 129, 70), (43, 70, 129), (43, 129, 257), (43, 300, 257), (2, 257, 64), (130, 64, 64)])
def test_batches(batch, rows, cols):
    """Equal matrices in one call: each as near as alone, whatever size of tile their number leads to."""
    say("orthogonalise a batch", batch, rows, cols)
    g = torch.stack([matrix(rows, cols, "few", i) for i in range(batch)]).cuda()
    got = gq().orthogonalise(g)
    for i in (0, 1, batch // 2, batch - 1):
        check(got[i], g[i])


@pytest.mark.parametrize("rows,cols", [(4096, 4096), (1100, 4500), (2100, 1000)])
def test_large_matrices(rows, cols):
    """The largest tiles, and splits of long sums: sampled rows of the result of 64 bits on the GPU."""
    say("orthogonalise large", rows, cols)
    g = torch.randn(rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(rows))
    got = gq().orthogonalise(g).double()
    x = g.double() if rows <= cols else g.double().T
    x = x / torch.linalg.matrix_norm(x)
    a, b, c = layers.QUINTIC
    for _ in range(5):
        p = x @ x.T.contiguous()
        x = a * x + (b * p + c * (p @ p)) @ x
    x = x if rows <= cols else x.T
    # bf16's roundings are 1.7e-3 of the norm; the others less than that
    assert (got - x).norm() <= 2.0 ** -8 * x.norm()


@pytest.mark.parametrize("steps", [1, 2, 3, 10])
@pytest.mark.parametrize("coefficients", [layers.QUINTIC, (1.875, -1.25, 0.375), (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)])
def test_steps_and_coefficients(steps, coefficients):
    say("orthogonalise steps", steps, coefficients)
    for rows, cols in ((96, 130), (130, 96)):
        g = matrix(rows, cols, "normal", 3).cuda()
        check(gq().orthogonalise(g, steps=steps, coefficients=coefficients), g, steps, coefficients)


def test_scale_does_not_matter():
    """Powers of two give the same bits, from where squares underflow in fp32 to where they overflow."""
    say("orthogonalise scales")
    g = gq()
    x = matrix(70, 90, "heavy", 1).cuda()
    want = g.orthogonalise(x)
    for e in (-90, -40, 60, 120):
        assert torch.equal(g.orthogonalise(x * 2.0 ** e), want), e


def test_zeros_and_what_is_not_finite():
    """A matrix of zeros gives zeros; an infinity or NaN makes its own matrix NaN and no other."""
    say("orthogonalise zeros")
    g = gq()
    for rows, cols in ((40, 70), (70, 40)):
        x = torch.stack([matrix(rows, cols, "normal", i) for i in range(5)]).cuda()
        x[1] = 0
        x[2, 3, 5] = float("inf")
        x[4, rows - 1, cols - 1] = float("nan")
        got = g.orthogonalise(x)
        assert not got[1].any() and torch.isnan(got[2]).all() and torch.isnan(got[4]).all()
        check(got[0], x[0])
        check(got[3], x[3])
        assert torch.equal(got[0], g.orthogonalise(x[:1])[0])


def test_strides():
    """Matrices within wider ones, at any element's alignment; what lies around the results stays."""
    say("orthogonalise strides")
    g = gq()
    for rows, cols in ((50, 67), (67, 50)):
        wide = torch.randn(4, rows + 2, cols + 3, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
        x = wide[:, :rows, :cols]
        out = torch.full((4, rows + 1, cols + 5), 3.0, dtype=BF16, device="cuda")
        got = g.orthogonalise(x, out=out[:, :rows, :cols])
        assert torch.equal(got, g.orthogonalise(x.contiguous()))
        assert torch.all(out[:, rows:] == 3) and torch.all(out[:, :, cols:] == 3)
        every = g.orthogonalise(wide[::3, :rows, :cols])
        assert torch.equal(every[1], got[3])


def test_same_bits_again():
    say("orthogonalise again")
    g = gq()
    x = torch.randn(6, 130, 500, device="cuda")
    assert torch.equal(g.orthogonalise(x), g.orthogonalise(x))


def test_refusals():
    say("orthogonalise refusals")
    g = gq()
    x = torch.ones(4, 6, device="cuda")
    assert g.orthogonalise(torch.zeros(0, 4, 6, device="cuda")).shape == (0, 4, 6)
    assert g.orthogonalise(torch.zeros(0, 6, device="cuda")).shape == (0, 6)
    for call in (lambda: g.orthogonalise(x, steps=0), lambda: g.orthogonalise(x, steps=33), lambda: g.orthogonalise(x, coefficients=(9.0, 0.0, 0.0)),
                 lambda: g.orthogonalise(x, coefficients=(3.4445, 4.7750, 2.0315)), lambda: g.orthogonalise(x, coefficients=(float("nan"), 0.0, 0.0)),
                 lambda: g.orthogonalise(torch.ones(1, 70000, device="cuda")),
                 lambda: g.orthogonalise(torch.ones(30, device="cuda")[1:25].view(4, 6)),
                 lambda: g.orthogonalise(x.bfloat16(), out=x.bfloat16()[:1].expand(4, 6))):
        with pytest.raises(g.GQError):
            call()
    y = x.bfloat16()
    with pytest.raises(g.GQError):
        g.orthogonalise(y, out=y)
    for call in (lambda: g.orthogonalise(x.half()), lambda: g.orthogonalise(x.cpu()), lambda: g.orthogonalise(x, out=torch.zeros(4, 6, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: g.orthogonalise(x.T), lambda: g.orthogonalise(x[0]), lambda: g.orthogonalise(x, out=torch.zeros(6, 4, dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            call()
