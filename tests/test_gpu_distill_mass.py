"""Distillation from teachers whose entries do not sum to one: entries that are all unlikely, all
above one, or more or less than a whole distribution.  The loss, its gradient fused, apart and in
place, against the definition."""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu

SHAPES = [(4, 700, torch.float32), (4, 9001, torch.bfloat16), (140, 20011, torch.float32)]


def bits(t):
    t = torch.where(torch.isnan(t), torch.full_like(t, float("nan")), t)
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def check(z, ids, lps, tail, temperature=1.0):
    g = gq()
    rows, vocab = z.shape
    w = np.random.default_rng(1).random(rows).astype(np.float32) + 0.1
    zd, wd = z.cuda(), torch.from_numpy(w).cuda()
    args = (torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda(), temperature, tail)
    loss, grad = g.distill_loss(zd, *args, row_weight=wd)
    alone, stats = g.distill_loss(zd, *args)
    apart = g.distill_grad(zd, *args, stats, wd)
    place = zd.clone()
    g.distill_loss(place, *args, row_weight=wd, dlogits=place)
    assert torch.equal(bits(alone), bits(loss))
    assert torch.equal(bits(apart), bits(grad)) and torch.equal(bits(place), bits(grad))
    z64 = z.float().numpy().astype(np.float64)
    rl, rg, _ = lm.distill(z64, ids, lps, temperature, tail, w)
    # the sums' error in the logarithms, times the mass; one rounding of the result
    eps = (vocab / 256 + 64) * 2.0 ** -22
    p = np.exp(lps.astype(np.float64)).sum(1) if tail else np.ones(rows)
    got = loss.double().cpu().numpy()
    tol = 4 * temperature ** 2 * eps * (1 + p) + np.abs(rl) * 2.0 ** -22
    assert np.all(np.abs(got - rl) <= tol), (got, rl)
    q = np.exp(lm.log_softmax(z64, temperature))
    scale = (w * temperature)[:, None].astype(np.float64)
    tol = 2 * eps * (np.abs(rg) + scale * (1 + p)[:, None] * q) + 2.0 ** -125
    if z.dtype == torch.bfloat16:
        tol = tol + np.abs(rg) * 2.0 ** -8
    got = grad.double().cpu().numpy()
    bad = ~(np.abs(got - rg) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], rg[bad][:4])


def rows_of(rows, vocab, dtype, top, seed):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy(rng.standard_normal((rows, vocab)).astype(np.float32) * 2).to(dtype)
    ids = np.stack([rng.permutation(vocab)[:top] for _ in range(rows)]).astype(np.int32)
    return z, ids, rng


@pytest.mark.parametrize("rows,vocab,dtype", SHAPES)
@pytest.mark.parametrize("level", [-95.0, -120.0, -800.0, -1e6, 100.0, 900.0])
def test_entries_far_from_one(rows, vocab, dtype, level):
    """Without a tail p is divided by its sum, whatever the sum: the loss of log p + c is that of
    log p.  Row 1 has one entry (p = 1), row 2 padding among them."""
    say("distill mass", rows, vocab, dtype, level)
    z, ids, rng = rows_of(rows, vocab, dtype, 6, 7)
    lps = (level + rng.standard_normal((rows, 6))).astype(np.float32)
    ids[1, 1:] = -1
    ids[2, 0], lps[2, 0] = -1, 0.0
    lps[3, 2] = -np.inf
    check(z, ids, lps, False)


def test_nothing_but_impossible_entries():
    say("distill all impossible")
    z, ids, _ = rows_of(2, 700, torch.float32, 3, 8)
    lps = np.full((2, 3), -np.inf, np.float32)
    lps[1, 1] = -2000.0
    check(z, ids, lps, False)


@pytest.mark.parametrize("rows,vocab,dtype", SHAPES)
@pytest.mark.parametrize("total", [0.4, 1.5, 7.0])
def test_tail_with_any_mass(rows, vocab, dtype, total):
    """The gradient is the loss's derivative also where the entries sum to more than one."""
    say("distill tail mass", rows, vocab, dtype, total)
    z, ids, rng = rows_of(rows, vocab, dtype, 6, 9)
    p = rng.random((rows, 6)) + 0.1
    check(z, ids, np.log(total * p / p.sum(1, keepdims=True)).astype(np.float32), True, 1.5)


@pytest.mark.parametrize("total", [0.4, 1.0, 1.5])
def test_tail_without_a_rest(total):
    """The whole vocabulary is taught: no entry is left for the bucket."""
    say("distill whole vocabulary", total)
    z, ids, rng = rows_of(4, 9, torch.float32, 9, 10)
    p = rng.random((4, 9)) + 0.1
    check(z, ids, np.log(total * p / p.sum(1, keepdims=True)).astype(np.float32), True, 1.5)
