"""The autograd functions over the language-model operators, and the example that runs them
together with the gradients' exchange."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_mx_linear_runs_the_formulas(dtype):
    from allreduce_compatible_gradient_amd import lm
    say("mx_linear", dtype)
    g = gq()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(70, 130, device="cuda", generator=gen).to(dtype).requires_grad_()
    w = torch.randn(90, 130, device="cuda", generator=gen).requires_grad_()
    b = torch.randn(90, device="cuda", generator=gen).requires_grad_()
    y = lm.mx_linear(x, w, b, seed=7, worker=2)
    dy = torch.randn(70, 90, device="cuda", generator=gen).to(dtype)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    assert y.dtype == dx.dtype == dtype and dw.dtype == torch.float32
    vals = lambda t, **k: [None if q is None else g.mx_dequantize(q, g.F32).double()  # noqa: E731
                           for q in g.mx_quantize(t.detach(), by_cols=True, **k)]
    (vx, vxt), (vw, vwt) = vals(x), vals(w)
    vd, vdt = vals(dy, rounding=g.MX_STOCHASTIC, seed=7, worker=2)
    # fp32 sums of at most 130 products, one more addition for the bias, and the type's rounding
    for got, a, c, more in ((y, vx, vw, b.detach().double()), (dx, vd, vwt, 0.0), (dw, vdt, vxt, 0.0)):
        want = a @ c.T + more
        tol = (a.abs() @ c.abs().T + abs(more)) * 70 * 2.0 ** -24
        if got.dtype == torch.bfloat16:
            tol = tol + want.abs() * 2.0 ** -8
        assert bool(((got.detach().double() - want).abs() <= tol).all())
    assert torch.allclose(db, dy.float().sum(0))


def test_mx_linear_gradient_is_unbiased():
    """The mean of dX over seeds against dY times the packed weights: each of the n draws of an
    entry has a spread of at most its grid's spacing, a third of its block's scale of 6 at most."""
    from allreduce_compatible_gradient_amd import lm
    say("mx_linear unbiased")
    g = gq()
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(8, 64, device="cuda", generator=gen).requires_grad_()
    w = torch.randn(64, 64, device="cuda", generator=gen)
    dy = torch.randn(8, 64, device="cuda", generator=gen)
    n = 400
    mean = sum(torch.autograd.grad(lm.mx_linear(x, w, seed=s), x, dy)[0].double() for s in range(n)) / n
    vwt = g.mx_dequantize(g.mx_quantize(w, by_cols=True)[1], g.F32).double()
    spacing = dy.abs().view(8, 2, 32).amax(2, keepdim=True).expand(8, 2, 32).reshape(8, 64).double() * 2 / 3
    spread = torch.sqrt((spacing ** 2 / 4) @ (vwt ** 2).T)      # a two-valued draw: half its spacing
    assert bool(((mean - dy.double() @ vwt.T).abs() <= 6 * spread / n ** 0.5).all())


def test_distill_autograd():
    from allreduce_compatible_gradient_amd import lm
    say("distill autograd")
    g = gq()
    gen = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(20, 333, device="cuda", generator=gen).requires_grad_()
    _, _, ids, lps = g.token_logprobs(torch.randn(20, 333, device="cuda", generator=gen),
                                      torch.zeros(20, dtype=torch.int64, device="cuda"), 9, 2.0)
    w = torch.rand(20, device="cuda", generator=gen)
    loss = lm.distill(z, ids, lps, 2.0, True)
    (d,) = torch.autograd.grad((loss * w).sum(), z)
    loss2, d2 = g.distill_loss(z.detach(), ids, lps, 2.0, True, row_weight=w)
    assert torch.equal(d, d2) and torch.equal(loss.detach(), loss2)


def test_example_learns():
    import importlib.util
    import os
    say("example")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_mx.py")
    spec = importlib.util.spec_from_file_location("distill_mx", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, entropy = ex.run(steps=30, workers=3, tokens=256, vocab=1031, say=None)
    assert all(np.isfinite(losses)) and entropy > 0
    assert losses[-1] < 0.7 * losses[0], losses
