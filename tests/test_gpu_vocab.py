"""Log probabilities and distillation on the GPU against the 64-bit definitions.

Tolerances: a thread adds vocab / 256 terms in turn and a few dozen joins follow, each rounding
by 2^-24 at most, and a term's own error is a few 2^-24 times its exponent: EPS(vocab) below is
twice that, relative to a softmax sum, and absolute for its logarithm."""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu


def EPS(vocab):
    return (vocab / 256 + 64) * 2.0 ** -22


def _logits(rows, vocab, dtype, seed, ties=False):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((rows, vocab)) * 3
    z[np.arange(rows), rng.integers(0, vocab, rows)] += 8
    if ties:
        z = np.round(z)
    return torch.from_numpy(z.astype(np.float32)).to(dtype)


def _check_logprobs(z, tokens, top, temperature=1.0, zd=None):
    g = gq()
    vocab = z.shape[1]
    lp, h, ids, lps = g.token_logprobs(zd if zd is not None else z.cuda(), torch.tensor(tokens).cuda(), top, temperature)
    rlp, rh, rids, rlps = lm.logprobs(z.float().numpy(), tokens, top, temperature)
    eps = EPS(vocab)
    lp, h = lp.cpu().numpy(), h.cpu().numpy()
    with np.errstate(invalid="ignore"):
        close = lambda a, b, e: np.all((a == b) | (np.isnan(a) & np.isnan(b)) | (np.abs(a - b) <= e))  # noqa: E731
        assert close(lp, rlp, eps + np.abs(rlp) * 2.0 ** -22), (lp, rlp)
        assert close(h, rh, eps * (1 + np.abs(rh))), (h, rh)
        if top:
            assert np.array_equal(ids.cpu().numpy(), rids)
            assert close(lps.cpu().numpy(), rlps, eps + np.abs(rlps) * 2.0 ** -22)


@pytest.mark.parametrize("rows,vocab", [(1, 1), (1, 2), (2, 7), (3, 8), (4, 100), (5, 2047), (3, 2049),
                                        (2, 8193), (1, 50257), (600, 1031), (1100, 257)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs(rows, vocab, dtype):
    say("logprobs", rows, vocab, dtype)
    z = _logits(rows, vocab, dtype, rows + vocab)
    tokens = np.random.default_rng(0).integers(0, vocab, rows)
    for top in sorted({0, 1, min(5, vocab), min(128, vocab)}):
        _check_logprobs(z, tokens, top)
    _check_logprobs(z, tokens, min(3, vocab), 0.3)


@pytest.mark.parametrize("vocab,rows", [(300, 2), (5000, 3), (131072, 1), (140001, 1)])
def test_logprobs_ties(vocab, rows):
    """More equal entries than there are places: the lowest indices, in order."""
    say("logprobs ties", vocab, rows)
    z = _logits(rows, vocab, torch.bfloat16, 3, ties=True)
    tokens = np.zeros(rows, np.int64)
    _check_logprobs(z, tokens, 100)
    z[0] = 1.5
    _check_logprobs(z, tokens, 64)
    z[0, ::3] = -0.0
    z[0, 1::3] = 0.0
    z[0, 2::3] = -1
    _check_logprobs(z, tokens, 17)


@pytest.mark.parametrize("vocab,top", [(50257, 20), (140001, 128), (200000, 128)])
def test_logprobs_largest_together(vocab, top):
    """The largest entries next to each other, in one of the slices of a row that is joined from
    many, or spread so that every slice has as many."""
    say("logprobs together", vocab, top)
    z = torch.zeros(3, vocab)
    z[0] = torch.arange(vocab) * 1e-3
    z[1] = -torch.arange(vocab) * 1e-3
    z[2, :: vocab // 997] = torch.arange(len(z[2, :: vocab // 997])) % 7 * 1.0
    _check_logprobs(z, np.zeros(3, np.int64), top)


@pytest.mark.parametrize("rows", [8, 1200])
def test_logprobs_masks(rows):
    """Rows that a mask leaves nothing or one entry, lowest finite values, infinities and NaN."""
    say("logprobs masks", rows)
    vocab = 700
    low = torch.finfo(torch.float32).min
    z = _logits(rows, vocab, torch.float32, 11)
    z[0] = float("-inf")
    z[1] = float("-inf")
    z[1, 333] = 2.5
    z[2] = low
    z[3, 50:] = low
    z[4, ::2] = float("-inf")
    z[5, 77] = float("nan")
    z[6, 78] = float("inf")
    z[7, 5] = 3e38
    tokens = np.full(rows, 333, np.int64)
    tokens[4], tokens[3], tokens[2] = 4, 60, 5
    _check_logprobs(z, tokens, 20)
    tokens[:3] = -1, vocab, -100                # no token: 0
    _check_logprobs(z, tokens, 0)


def test_logprobs_strided_rows():
    say("logprobs strides")
    wide = _logits(9, 1111, torch.bfloat16, 5)
    _check_logprobs(wide[:, :1003], np.arange(9), 7, zd=wide.cuda()[:, :1003])


# ----------------------------------------------------------------------------- distillation
def _teacher(z, top, temperature, seed):
    rng = np.random.default_rng(seed)
    t = z.float().numpy() + rng.standard_normal(z.shape)
    lt = lm.log_softmax(t, temperature)
    ids = np.argsort(-lt, 1, kind="stable")[:, :top]
    return ids.astype(np.int32), np.take_along_axis(lt, ids, 1).astype(np.float32)


def _check_distill(z, ids, lps, temperature, tail, zd=None):
    g = gq()
    rows, vocab = z.shape
    zd = zd if zd is not None else z.cuda()
    w = np.random.default_rng(1).random(rows).astype(np.float32) + 0.1
    args = (torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda(), temperature, tail)
    wd = torch.from_numpy(w).cuda()
    loss, grad = g.distill_loss(zd, *args, row_weight=wd)
    loss2, stats = g.distill_loss(zd, *args)
    grad2 = g.distill_grad(zd, *args, stats, wd)
    assert torch.equal(torch.nan_to_num(loss), torch.nan_to_num(loss2))
    assert torch.equal(torch.nan_to_num(grad), torch.nan_to_num(grad2))
    place = zd.clone()
    g.distill_loss(place, *args, row_weight=wd, dlogits=place)
    assert torch.equal(torch.nan_to_num(place), torch.nan_to_num(grad))
    rl, rg, rest = lm.distill(z.float().numpy(), ids, lps, temperature, tail, w)
    eps, top = EPS(vocab), ids.shape[1]
    p_r, q_r = rest[:, 0], rest[:, 1]
    with np.errstate(all="ignore"):
        ratio = np.where(p_r > 0, np.abs(np.log(p_r / q_r)), 0.0)
        # the sum of p rounds by top 2^-23, which p_R has as an absolute error
        tol = temperature ** 2 * (eps * (2 + ratio) + top * 2.0 ** -23 * (2 + ratio)) + np.abs(rl) * 2.0 ** -22
        got = loss.cpu().numpy()
        assert np.all((got == rl) | (np.isnan(got) & np.isnan(rl)) | (np.abs(got - rl) <= tol)), (got, rl)
        q = np.exp(lm.log_softmax(z.float().numpy(), temperature))
        scale = (w * temperature)[:, None]
        tol = scale * ((q + np.abs(rg) / scale) * eps + q * np.where(p_r > 0, p_r / q_r, 0)[:, None] * 2 * eps
                       + q * np.where(q_r > 0, top * 2.0 ** -22 / q_r, 0)[:, None] + 2.0 ** -22 * (np.abs(rg) / scale + q))
        if z.dtype == torch.bfloat16:
            tol = tol + np.abs(rg) * 2.0 ** -8
        got = grad.float().cpu().numpy()
        # below the type's normal range a gradient rounds by its smallest step
        tol = tol + 2.0 ** -126
        bad = ~((got == rg) | (np.isnan(got) & np.isnan(rg)) | (np.abs(got - rg) <= tol))
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], rg[bad][:4])


@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (2, 9, 9), (3, 100, 7), (5, 2049, 16), (2, 8200, 128),
                                            (1, 50257, 33), (1100, 520, 20), (2, 140001, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tail", [False, True])
def test_distill(rows, vocab, top, dtype, tail):
    say("distill", rows, vocab, top, dtype, tail)
    z = _logits(rows, vocab, dtype, rows + vocab + top)
    for temperature in (1.0, 2.5):
        _check_distill(z, *_teacher(z, top, temperature, 3), temperature, tail)


@pytest.mark.parametrize("rows", [6, 1200])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_padding_repeats_and_masks(rows, tail):
    say("distill padding", rows, tail)
    vocab = 900
    z = _logits(rows, vocab, torch.float32, 4)
    ids, lps = _teacher(z, 12, 1.0, 5)
    ids[0] = -1                                  # taught nothing
    ids[1, 4:] = -1
    ids[2, 3], ids[2, 7] = ids[2, 0], vocab      # occurs again; outside
    lps[3, 5] = -np.inf                          # p = 0
    z[4] = float("-inf")
    z[4, ids[4]] = torch.randn(12)               # only taught entries are left
    lps[4] = lm.log_softmax(lps[4:5], 1.0)[0]
    z[5, 100:200] = float("-inf")
    ids[5, 0] = 1
    _check_distill(z, ids, lps, 1.0, tail)


def test_distill_masked_student_and_nan():
    say("distill masked")
    z = torch.zeros(4, 50)
    z[0] = float("-inf")                         # no probability anywhere: an infinite loss, gradient -p
    z[1, 3] = float("nan")
    z[2, 7] = float("-inf")                      # a taught entry without probability
    z[3, 4] = float("nan")                       # taught nothing: 0 whatever the logits are
    ids = np.array([[1, 2], [1, 2], [7, 2], [-1, -1]], np.int32)
    lps = np.log(np.array([[0.5, 0.5]] * 4, np.float32))
    g = gq()
    for tail in (False, True):
        loss, grad = g.distill_loss(z.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda(), 1.0, tail,
                                    row_weight=torch.ones(4).cuda())
        loss, grad = loss.cpu(), grad.cpu()
        assert loss[0] == float("inf") and torch.isnan(loss[1]) and loss[2] == float("inf") and loss[3] == 0
        assert torch.allclose(grad[0, [1, 2]], torch.tensor([-0.5, -0.5])) and float(grad[0].abs().sum()) == 1
        assert torch.isnan(grad[1, 0]) and not bool(grad[3].any())
        assert abs(float(grad[2, 7]) + 0.5) < 1e-6


def test_distill_strided_rows():
    say("distill strides")
    wide = _logits(9, 1111, torch.bfloat16, 5)
    z = wide[:, :1003]
    _check_distill(z, *_teacher(z, 10, 1.0, 6), 1.0, True, zd=wide.cuda()[:, :1003])
    g = gq()
    ids, lps = _teacher(z, 10, 1.0, 6)
    out = torch.full((9, 1100), 5.0, dtype=torch.bfloat16, device="cuda")
    args = (torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda())
    _, grad = g.distill_loss(z.cuda(), *args, row_weight=torch.ones(9).cuda())
    g.distill_loss(z.cuda(), *args, dlogits=out[:, :1003])
    assert torch.equal(out[:, :1003], grad) and bool((out[:, 1003:] == 5).all())


def test_distill_gradient_against_differences():
    """Central differences of the loss the library itself computes, in fp32 with a step of 2^-6:
    the quotient's rounding is a few 2^-24 of the loss over the step, its truncation h^2 / 6."""
    say("distill differences")
    g = gq()
    z = _logits(1, 40, torch.float32, 9)
    ids, lps = _teacher(z, 6, 1.5, 2)
    args = (torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda(), 1.5, True)
    loss, grad = g.distill_loss(z.cuda(), *args, row_weight=torch.ones(1).cuda())
    h = 2.0 ** -6
    step = torch.eye(40) * h
    many = lambda s: g.distill_loss((z + s * step).cuda(), args[0].expand(40, -1).contiguous(),  # noqa: E731
                                    args[1].expand(40, -1).contiguous(), 1.5, True)[0]
    d = (many(1) - many(-1)).double() / (2 * h)
    tol = (float(loss) + 8) * 16 * 2.0 ** -24 / h + h * h
    assert float((d.cpu() - grad[0].double().cpu()).abs().max()) <= tol


def test_logprobs_feed_distillation():
    """A teacher's answers as they come out of token_logprobs: its own logits lose nothing."""
    say("logprobs to distill")
    g = gq()
    z = _logits(64, 3001, torch.bfloat16, 12).cuda()
    _, _, ids, lps = g.token_logprobs(z, torch.zeros(64, dtype=torch.int64).cuda(), 32, 2.0)
    loss, grad = g.distill_loss(z, ids, lps, 2.0, True, row_weight=torch.ones(64).cuda())
    # log p - log q and p - q are the roundings of two passes
    assert float(loss.abs().max()) <= 4 * 4 * EPS(3001) and float(grad.abs().max()) <= 2 * 4 * EPS(3001)


def test_vocab_side_stream_and_graph():
    say("vocab graph")
    g = gq()
    ctx = g.Context()
    z = torch.randn(3, 9001, device="cuda")
    ids = torch.randint(0, 9001, (3, 8), dtype=torch.int32, device="cuda")
    lps = torch.full((3, 8), -3.0, device="cuda")
    tokens = torch.zeros(3, dtype=torch.int64, device="cuda")
    w = torch.ones(3, device="cuda")
    grad = torch.empty_like(z)
    out = g.token_logprobs(z, tokens, 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def both():
        g.token_logprobs(z, tokens, 9, out=out, ctx=ctx)
        return g.distill_loss(z, ids, lps, 1.0, True, row_weight=w, dlogits=grad, ctx=ctx)[0]

    with torch.cuda.stream(s):
        both()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        loss = both()
    for i in range(3):
        z.copy_(torch.randn(3, 9001) * 3)
        want = g.token_logprobs(z, tokens, 9)
        wl, wg = g.distill_loss(z, ids, lps, 1.0, True, row_weight=w)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        assert torch.equal(loss, wl) and torch.equal(grad, wg), i


def test_refusals():
    say("vocab refusals")
    g = gq()
    z = torch.zeros(3, 50, device="cuda")
    tokens = torch.zeros(3, dtype=torch.int64, device="cuda")
    ids = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    lps = torch.zeros(3, 4, device="cuda")
    for kw in (dict(top=51), dict(top=-1), dict(temperature=0.0), dict(temperature=float("nan"))):
        with pytest.raises(g.GQError) as e:
            g.token_logprobs(z, tokens, **kw)
        assert e.value.code == g.EINVAL
    with pytest.raises(g.GQError):
        g.token_logprobs(torch.zeros(2, 300, device="cuda"), tokens[:2], top=129)
    with pytest.raises(TypeError):
        g.token_logprobs(z, tokens.int())
    with pytest.raises(TypeError):
        g.token_logprobs(z.half(), tokens)
    with pytest.raises(ValueError):
        g.token_logprobs(z, tokens[:2])
    with pytest.raises(ValueError):
        g.token_logprobs(z.T, tokens)
    with pytest.raises(g.GQError):
        g.distill_loss(z, ids, lps, temperature=-1.0)
    with pytest.raises(g.GQError):
        g.distill_loss(z, torch.zeros(3, 129, dtype=torch.int32, device="cuda"), torch.zeros(3, 129, device="cuda"))
    with pytest.raises(ValueError):
        g.distill_loss(z, ids, lps[:2])
    with pytest.raises(ValueError):
        g.distill_loss(z, ids, lps, row_weight=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        g.distill_loss(z, ids, lps, dlogits=torch.empty(3, 49, device="cuda"))
    lib, ctx = g._lib, g.context()
    buf = torch.empty(64, device="cuda")
    call = lambda **k: lib.gq_distill_grad(ctx.handle, z.data_ptr(), 0, 3, 50, k.get("ld", 50), ids.data_ptr(),  # noqa: E731
                                           lps.data_ptr(), 4, 1.0, k.get("tail", 0), k.get("stats", buf.data_ptr()),
                                           None, k.get("d", z.data_ptr()), k.get("ldd", 50), None)
    assert call(ld=49) == g.EINVAL and call(tail=2) == g.EINVAL and call(stats=None) == g.EINVAL
    assert call(ldd=49) == g.EINVAL and call(ldd=60) == g.EINVAL and call(d=z.data_ptr() + 8) == g.EALIGN
