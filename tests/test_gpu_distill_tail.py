"""Distillation with one bucket for the rest where the student has next to nothing left for it: the
bucket's logarithm and its gradient stay numbers when q_R itself is below every type's range.

Tolerances: `eps` as for the row's sums (vocab / 256 adds in turn and a few dozen joins); an
exponential's error is 2^-23 of its exponent, and a gradient's factors round a few times more."""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu

# held by 256 threads; in slices; held by 512 threads
SHAPES = [(3, 700, torch.float32), (2, 9001, torch.bfloat16), (3, 70001, torch.float32), (140, 20011, torch.float32)]


def bits(t):
    t = torch.where(torch.isnan(t), torch.full_like(t, float("nan")), t)
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def check(z, ids, lps, temperature=1.0):
    """Against the definition; the gradient apart and in place has the same bits, NaN or not."""
    g = gq()
    rows, vocab = z.shape
    w = np.random.default_rng(1).random(rows).astype(np.float32) + 0.1
    zd, wd = z.cuda(), torch.from_numpy(w).cuda()
    args = (torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda(), temperature, True)
    loss, grad = g.distill_loss(zd, *args, row_weight=wd)
    alone, stats = g.distill_loss(zd, *args)
    apart = g.distill_grad(zd, *args, stats, wd)
    place = zd.clone()
    g.distill_loss(place, *args, row_weight=wd, dlogits=place)
    assert torch.equal(bits(alone), bits(loss))
    assert torch.equal(bits(apart), bits(grad)) and torch.equal(bits(place), bits(grad))
    z64 = z.float().numpy().astype(np.float64)
    rl, rg, _ = lm.distill(z64, ids, lps, temperature, True, w)
    eps = (vocab / 256 + 64) * 2.0 ** -22
    got = loss.double().cpu().numpy()
    with np.errstate(all="ignore"):
        # the logarithms of two sums, then one rounding
        tol = 4 * temperature ** 2 * eps + np.abs(rl) * 2.0 ** -22
        assert np.all((got == rl) | (np.abs(got - rl) <= tol)), (got, rl)
    scale = (w * temperature)[:, None].astype(np.float64)
    taught = np.zeros(z.shape, bool)
    for i in range(rows):
        taught[i, ids[i][lm.taught_entries(ids[i], vocab)]] = True
    low = np.where(taught, -np.inf, z64).max(1, keepdims=True)
    depth = np.where(taught, 0.0, (low - z64) / temperature)     # of R's entries below their largest
    q = np.exp(lm.log_softmax(z64, temperature))
    tol = np.abs(rg) * (2 * eps + depth * 2.0 ** -21) + scale * (taught * q * eps + 2.0 ** -125)
    if z.dtype == torch.bfloat16:
        tol = tol + np.abs(rg) * 2.0 ** -8
    got = grad.double().cpu().numpy()
    bad = ~(np.abs(got - rg) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], rg[bad][:4])
    return loss, grad


def rows_with_gap(rows, vocab, dtype, gap, temperature, p):
    """Logits of spread 2 T whose taught entries stand `gap` T above the rest; sum p = `p`."""
    rng = np.random.default_rng(rows + vocab)
    z = rng.standard_normal((rows, vocab)) * 2 * temperature
    ids = np.stack([rng.permutation(vocab)[:5] for _ in range(rows)]).astype(np.int32)
    np.put_along_axis(z, ids.astype(np.int64), gap * temperature + rng.standard_normal((rows, 5)), 1)
    share = rng.random((rows, 5)) + 0.2
    lps = np.log(p * share / share.sum(1, keepdims=True)).astype(np.float32)
    return torch.from_numpy(z.astype(np.float32)).to(dtype), ids, lps


@pytest.mark.parametrize("rows,vocab,dtype", SHAPES)
@pytest.mark.parametrize("gap", [100.0, 1000.0])
@pytest.mark.parametrize("temperature", [1.0, 0.125])
def test_rest_far_below_the_taught_entries(rows, vocab, dtype, gap, temperature):
    say("tail gap", rows, vocab, dtype, gap, temperature)
    z, ids, lps = rows_with_gap(rows, vocab, dtype, gap, temperature, 0.9)
    loss, grad = check(z, ids, lps, temperature)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad.float()).all())


@pytest.mark.parametrize("vocab", [700, 9001])
@pytest.mark.parametrize("mask", [-1e4, torch.finfo(torch.float32).min])
def test_rest_masked_with_finite_values(vocab, mask):
    """The rest masked with a finite value: with mass for it the loss is large and finite and the
    mass is spread evenly; a mass that is the sum's rounding counts as none."""
    say("tail finite mask", vocab, mask)
    z, ids, lps = rows_with_gap(2, vocab, torch.float32, 0.0, 1.0, 0.9)
    lps[1] = np.log(np.full(5, 0.2)).astype(np.float32)          # sums to 1 within fp32's rounding
    taught = np.zeros(z.shape, bool)
    np.put_along_axis(taught, ids.astype(np.int64), True, 1)
    z[torch.from_numpy(~taught)] = mask
    loss, grad = check(z, ids, lps)
    assert bool(torch.isfinite(loss).all()) and float(loss[1]) < 10.0
    rest = grad.cpu()[0][torch.from_numpy(~taught[0])]
    assert float(rest.max()) < 0 and float(rest.max()) == float(rest.min())


def test_rest_masked_with_infinity():
    say("tail infinite mask")
    z, ids, lps = rows_with_gap(2, 700, torch.float32, 0.0, 1.0, 0.9)
    lps[1] = np.log(np.full(5, 0.2)).astype(np.float32)
    taught = np.zeros(z.shape, bool)
    np.put_along_axis(taught, ids.astype(np.int64), True, 1)
    z[torch.from_numpy(~taught)] = -np.inf
    g = gq()
    loss, grad = g.distill_loss(z.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda(), 1.0, True,
                                row_weight=torch.ones(2).cuda())
    assert float(loss[0]) == float("inf") and float(loss[1]) < 10.0
    assert bool((grad.cpu()[torch.from_numpy(~taught)] == 0).all())
