"""The operators around a model's layers under autograd and together: formulas, views and empty batches,
graphs, two streams, and the example that runs them all."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import layers
from tests.gpu_helpers import gq, host, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def values(q):
    """The 64-bit values of a packed 8-bit matrix."""
    return q.codes[:, :q.cols].double() * q.scales.double()[:, None]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_int_linear_runs_the_formulas(dtype):
    from allreduce_compatible_gradient_amd import lm
    say("int_linear", dtype)
    g = gq()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(70, 130, device="cuda", generator=gen).to(dtype).requires_grad_()
    w = torch.randn(90, 130, device="cuda", generator=gen).requires_grad_()
    b = torch.randn(90, device="cuda", generator=gen).requires_grad_()
    y = lm.int_linear(x, w, b, seed=7, worker=2)
    dy = torch.randn(70, 90, device="cuda", generator=gen).to(dtype)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    assert y.dtype == dx.dtype == dtype and dw.dtype == torch.float32
    vals = lambda t, **k: [values(q) for q in g.int_quantize(t.detach(), by_cols=True, **k)]  # noqa: E731
    (vx, vxt), (vw, vwt) = vals(x), vals(w)
    vd, vdt = vals(dy, rounding=g.INT_STOCHASTIC, seed=7, worker=2)
    # exact sums; three roundings of the product, one of the sum with the bias, and the type's.  The 64-bit
    # values here are sums of at most 130 products, each step off by at most 2^-53 of their magnitudes'
    # sum: below 2^-45 of it (codes whose sum is 0 have a 0 here that is not)
    for got, a, c, more in ((y, vx, vw, b.detach().double()), (dx, vd, vwt, 0.0), (dw, vdt, vxt, 0.0)):
        product = a @ c.T
        want = product + more
        tol = (product.abs() * 3 + want.abs()) * 2.0 ** -24 * 1.01 + (a.abs() @ c.abs().T) * 2.0 ** -45
        if got.dtype == BF16:
            tol = tol + want.abs() * 2.0 ** -8
        assert bool(((got.detach().double() - want).abs() <= tol).all())
    assert torch.allclose(db, dy.float().sum(0))


def test_int_linear_gradient_is_unbiased():
    """The mean of dX over seeds against dY times the packed weights: a draw's spread is at most half
    its row's scale; six of them over the seeds."""
    from allreduce_compatible_gradient_amd import lm
    say("int_linear unbiased")
    g = gq()
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(8, 64, device="cuda", generator=gen).requires_grad_()
    w = torch.randn(64, 64, device="cuda", generator=gen)
    dy = torch.randn(8, 64, device="cuda", generator=gen)
    n = 400
    mean = sum(torch.autograd.grad(lm.int_linear(x, w, seed=s), x, dy)[0].double() for s in range(n)) / n
    vwt = values(g.int_quantize(w, by_cols=True)[1])
    spread = dy.abs().amax(1, keepdim=True).double() / 127 / 2 * vwt.square().sum(1).sqrt()
    # and the roundings of scale and quotient
    slack = 2.0 ** -20 * (dy.double().abs() @ vwt.abs().T)
    assert bool(((mean - dy.double() @ vwt.T).abs() <= 6 * spread / n ** 0.5 + slack).all())


@pytest.mark.parametrize("need", [(True, False), (False, True), (True, True)])
def test_int_linear_views_and_parts(need):
    """Views at any element, gradients of a cat, each gradient alone: the same bits as from copies."""
    from allreduce_compatible_gradient_amd import lm
    say("int_linear views", need)
    base_x, base_w = torch.randn(31 * 70 + 3, device="cuda"), torch.randn(33, 75, device="cuda")
    outs = []
    for copy in (False, True):
        x, w = base_x[3:].view(31, 70), base_w[1:, 2:72]
        x, w = [(t.clone() if copy else t).detach().requires_grad_(n) for t, n in zip((x, w), need)]
        y = lm.int_linear(x, w, seed=3)
        z = torch.cat([y, y * 2], 1)
        outs.append([y.detach()] + list(torch.autograd.grad((z * torch.arange(64, device="cuda")).sum(), [t for t in (x, w) if t.requires_grad])))
    assert all(torch.equal(p, q) for p, q in zip(*outs))


def test_empty_batches():
    from allreduce_compatible_gradient_amd import lm
    say("empty batches")
    w = torch.randn(9, 20, device="cuda", requires_grad=True)
    x = torch.zeros(0, 20, device="cuda", requires_grad=True)
    y = lm.int_linear(x, w)
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    assert y.shape == (0, 9) and dx.shape == (0, 20) and not dw.any()
    t = torch.randn(9, 20, device="cuda", requires_grad=True)
    e = lm.embedding(t, torch.zeros(0, 3, dtype=torch.int64, device="cuda"))
    (dt,) = torch.autograd.grad(e.sum(), t)
    assert e.shape == (0, 3, 20) and not dt.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embedding_autograd(dtype):
    from allreduce_compatible_gradient_amd import lm
    say("embedding autograd", dtype)
    t = torch.randn(50, 24, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dtype).requires_grad_()
    ids = torch.randint(-2, 52, (7, 11), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    w = torch.randn(7, 11, 24, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    out = lm.embedding(t, ids, scale=3.0, out_dtype=torch.float32)
    assert out.shape == (7, 11, 24) and out.dtype == torch.float32
    (d,) = torch.autograd.grad((out * w).sum(), t)
    assert d.dtype == dtype
    want, mass, count = layers.embedding_grad(w.view(-1, 24).cpu().numpy(), ids.view(-1).cpu().numpy(), 50, 3.0)
    bound = mass * (count[:, None] + 1) * 2.0 ** -24
    if dtype == BF16:
        bound = bound + np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -8)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= bound * (1 + 1e-5))


def test_differentiable_once():
    from allreduce_compatible_gradient_amd import lm
    say("differentiable once")
    t, w = torch.randn(6, 8, device="cuda", requires_grad=True), torch.randn(5, 8, device="cuda", requires_grad=True)
    ids = torch.tensor([1, 2], device="cuda")
    for f, leaf in ((lambda: lm.embedding(t, ids).square().sum(), t), (lambda: lm.int_linear(t, w).square().sum(), w)):
        (d,) = torch.autograd.grad(f(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            d.sum().backward()


def everything(g, s, ctx):
    """One run of the operators together, as a training step uses them, onto given outputs."""
    g.embedding(s["table"], s["ids"], scale=2.0, out=s["x"], ctx=ctx)
    q, _ = g.int_quantize(s["w"], out=s["qw"], ctx=ctx)
    g.int_matmul(s["x"], q, out_dtype=g.F32, out=s["y"], ctx=ctx)
    d, dt = g.int_quantize(s["y"], g.INT_STOCHASTIC, 5, by_cols=True, out=s["qd"], out_t=s["qdt"], ctx=ctx)
    _, xt = g.int_quantize(s["x"], by_rows=False, by_cols=True, out_t=s["qxt"], ctx=ctx)
    g.int_matmul(dt, xt, out_dtype=g.F32, out=s["dw"], ctx=ctx)
    g.embedding_grad(s["x"], s["ids"], s["table"].shape[0], out=s["dtable"], ctx=ctx)
    g.orthogonalise(s["dw"], out=s["u"], ctx=ctx)
    g.orthogonalise(s["dtable"], out=s["ut"], ctx=ctx)
    return [s[k] for k in ("x", "y", "dw", "dtable", "u", "ut")]


def state(g, seed, tokens=300, vocab=700, dim=136, out=520):
    gen = torch.Generator("cuda").manual_seed(seed)
    e = lambda *shape, dtype=F32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    return dict(table=torch.randn(vocab, dim, device="cuda", generator=gen), w=torch.randn(out, dim, device="cuda", generator=gen),
                ids=torch.randint(-1, vocab // 5, (tokens,), device="cuda", generator=gen), x=e(tokens, dim), y=e(tokens, out),
                dw=e(out, dim), dtable=e(vocab, dim), u=e(out, dim, dtype=BF16), ut=e(vocab, dim, dtype=BF16),
                qw=g.IntTensor.empty(out, dim, "cuda"), qd=g.IntTensor.empty(tokens, out, "cuda"),
                qdt=g.IntTensor.empty(out, tokens, "cuda"), qxt=g.IntTensor.empty(dim, tokens, "cuda"))


def test_together_against_the_definitions():
    """Each result against the definition applied to what the call was given."""
    say("together")
    g = gq()
    s = state(g, 1)
    x, y, dw, dtable, u, ut = everything(g, s, None)
    ids = s["ids"].cpu().numpy()
    assert np.array_equal(host(x), layers.embedding(host(s["table"]), ids, 2.0).astype(np.float32))
    assert np.array_equal(host(s["qw"].codes), layers.quantize(host(s["w"]), 0)[0])
    qx = layers.quantize(host(x), 0)
    want, mag = layers.matmul(*qx, host(s["qw"].codes), host(s["qw"].scales))
    assert np.all(np.abs(host(y) - want) <= mag * 3.01 * 2.0 ** -24)
    want, mag = layers.matmul(host(s["qdt"].codes), host(s["qdt"].scales), host(s["qxt"].codes), host(s["qxt"].scales))
    assert np.all(np.abs(host(dw) - want) <= mag * 3.01 * 2.0 ** -24)
    want, mass, count = layers.embedding_grad(host(x), ids, 700, 1.0)
    assert np.all(np.abs(host(dtable) - want) <= mass * (count[:, None] + 1) * 2.0 ** -24)
    for a, b in ((dw, u), (dtable, ut)):
        exact = layers.orthogonalise(host(a))
        own = np.linalg.norm(layers.orthogonalise_rounded(host(a)) - exact)
        assert np.linalg.norm(b.double().cpu().numpy() - exact) <= 1.5 * own + 2.0 ** -14 * np.linalg.norm(exact)


def test_in_a_graph():
    """Captured once, replayed with other inputs, the program's own work on the default context between."""
    say("graph")
    g = gq()
    ctx = g.Context()
    s = state(g, 2)
    everything(g, s, ctx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        everything(g, s, ctx)
    for seed in (3, 4, 5):
        other = state(g, seed)
        want = [t.clone() for t in everything(g, other, None)]
        for k in ("table", "w", "ids"):
            s[k].copy_(other[k])
        graph.replay()
        torch.cuda.synchronize()
        for k, w in zip(("x", "y", "dw", "dtable", "u", "ut"), want):
            assert torch.equal(s[k], w), (seed, k)
    del graph


def test_on_two_streams():
    """A context each: what runs at the same time does not share scratch memory."""
    say("two streams")
    g = gq()
    states, want = [], []
    for seed in (6, 7):
        states.append(state(g, seed, tokens=2000, vocab=3001, dim=200, out=900))
        want.append([t.clone() for t in everything(g, states[-1], None)])
    streams, contexts = [torch.cuda.Stream() for _ in states], [g.Context() for _ in states]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, stream, ctx in zip(states, streams, contexts):
            with torch.cuda.stream(stream):
                everything(g, s, ctx)
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        for k, t in zip(("x", "y", "dw", "dtable", "u", "ut"), w):
            assert torch.equal(s[k], t), k


def test_example_runs():
    say("train_tokens")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_tokens.py")
    spec = importlib.util.spec_from_file_location("train_tokens", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, grads = ex.run(steps=6, workers=2, tokens=200, vocab=1031, say=None)
    assert all(np.isfinite(losses)) and len(losses) == 6
    assert all(bool(torch.isfinite(d).all()) and bool(d.any()) for d in grads)
