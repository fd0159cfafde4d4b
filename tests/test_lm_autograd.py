"""The autograd functions' own work -- what they hand to the library, and to autograd -- on a stand-in
for the binding that computes the operators with torch in 64 bits and refuses what the library
refuses (CPU only; the products are not rounded to 4 bits)."""
import pytest
import torch

from allreduce_compatible_gradient_amd import gq, lm


class Refused(Exception):
    pass


def need(t, strided=False):
    """The library's conditions on a tensor: rows without gaps, on 16 bytes."""
    if t is None:
        return
    rows = t.dim() == 2 and strided and (t.stride(1) == 1 or t.shape[1] <= 1) and \
        (t.shape[0] <= 1 or t.stride(0) >= t.shape[1])
    if not (t.is_contiguous() or rows):
        raise Refused("rows with gaps")
    if t.data_ptr() % 16:
        raise Refused("not on 16 bytes")


@pytest.fixture
def calls(monkeypatch):
    """Installs the stand-in; the list of (function, keyword arguments) of the calls made."""
    made = []

    def mx_quantize(x, rounding=0, seed=0, worker=0, index_base=0, by_rows=True, by_cols=False, **kw):
        made.append(("mx_quantize", dict(kw, rounding=rounding, seed=seed, worker=worker)))
        need(x, strided=True)
        v = x.detach().double()
        return (v.clone() if by_rows else None), (v.T.contiguous() if by_cols else None)

    def mx_matmul(a, b, bias=None, out_dtype=gq.BF16, **kw):
        made.append(("mx_matmul", kw))
        need(bias)
        if a.shape[1] == 0 and a.shape[0] > 0:
            raise Refused("row length 0")
        if bias is not None and bias.dtype != torch.float32:
            raise Refused("bias")
        y = a @ b.T + (0.0 if bias is None else bias.double())
        return y.to(torch.float32 if out_dtype == gq.F32 else torch.bfloat16)

    def pieces(z, ids, lps, temperature, tail):
        assert not tail
        q = torch.softmax(z.double() / temperature, 1)
        p = torch.softmax(lps.double(), 1)
        return q, p, ids.long()

    def distill_loss(logits, ids, lps, temperature=1.0, tail=False, **kw):
        made.append(("distill_loss", kw))
        need(logits, strided=True), need(ids), need(lps)
        q, p, at = pieces(logits, ids, lps, temperature, tail)
        loss = temperature ** 2 * (p * (p.log() - q.gather(1, at).log())).sum(1)
        return loss.float(), torch.zeros(len(loss), 4)

    def distill_grad(logits, ids, lps, temperature, tail, stats, row_weight=None, **kw):
        made.append(("distill_grad", kw))
        need(logits, strided=True), need(ids), need(lps), need(stats), need(row_weight)
        q, p, at = pieces(logits, ids, lps, temperature, tail)
        return (row_weight.double()[:, None] * temperature * q.scatter_add(1, at, -p)).to(logits.dtype)

    for f in (mx_quantize, mx_matmul, distill_loss, distill_grad):
        monkeypatch.setattr(gq, f.__name__, f)
    return made


def parts(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def plain_distill(z, ids, lps, temperature):
    p = torch.softmax(lps.double(), 1)
    return temperature ** 2 * (p * (p.log() - torch.log_softmax(z.double() / temperature, 1).gather(1, ids.long()))).sum(1)


def test_gradients_that_start_anywhere(calls):
    """The gradient of a torch.cat is a view of the whole: contiguous, at any element."""
    w = parts(7, 9, seed=1).requires_grad_()
    x = [parts(5, 9, seed=2).requires_grad_(), parts(6, 9, seed=3).requires_grad_()]
    weight = parts(11, 7, seed=4)
    got = torch.autograd.grad((torch.cat([lm.mx_linear(t, w) for t in x]) * weight).sum(), [w] + x)
    want = torch.autograd.grad((torch.cat([t @ w.T for t in x]) * weight).sum(), [w] + x)
    assert all(torch.allclose(a, b, atol=1e-5) for a, b in zip(got, want))
    z = [parts(5, 33, seed=5).requires_grad_(), parts(7, 33, seed=6).requires_grad_()]
    ids = [torch.arange(3, dtype=torch.int32).expand(len(t), 3).contiguous() for t in z]
    lps = [parts(len(t), 3, seed=7) for t in z]
    weight = parts(12, seed=8)
    got = torch.autograd.grad((torch.cat([lm.distill(*a) for a in zip(z, ids, lps)]) * weight).sum(), z)
    want = torch.autograd.grad((torch.cat([plain_distill(*a, 1.0) for a in zip(z, ids, lps)]) * weight).sum(), z)
    assert all(torch.allclose(a, b, atol=1e-5) for a, b in zip(got, want))


def test_inputs_that_start_anywhere(calls):
    """Rows after the first of an odd length, transposed and strided views, pieces of a flat buffer."""
    flat = parts(1 + 63 + 7, seed=1)
    w, b = flat[1:64].view(7, 9).requires_grad_(), flat[64:].requires_grad_()
    whole = parts(9, 12, seed=2)
    for x in (parts(6, 9, seed=3)[1:], whole.T[:, :9], parts(6, 13, seed=4)[:, :9], parts(6, 13, seed=4)[:, 2:11],
              parts(9, seed=5).expand(4, 9)):
        x = x.detach().requires_grad_()
        assert torch.allclose(lm.mx_linear(x, w, b), x @ w.T + b, atol=1e-5)
        got = torch.autograd.grad(lm.mx_linear(x, w, b).sum(), (x, w, b))
        want = torch.autograd.grad((x @ w.T + b).sum(), (x, w, b))
        assert all(torch.allclose(p, q, atol=1e-5) for p, q in zip(got, want))
    ids = torch.arange(15, dtype=torch.int32).view(5, 3)
    for z in (parts(6, 33, seed=6)[1:], parts(33, 5, seed=7).T, parts(5, 40, seed=8)[:, 3:36]):
        z = z.detach().requires_grad_()
        teacher = (torch.cat([ids[:1], ids])[1:], parts(5, 4, seed=9)[:, 1:])
        got, = torch.autograd.grad(lm.distill(z, *teacher, 2.0).sum(), z)
        want, = torch.autograd.grad(plain_distill(z, *teacher, 2.0).sum(), z)
        assert torch.allclose(got, want, atol=1e-5)


@pytest.mark.parametrize("bias", [False, True])
def test_no_tokens(calls, bias):
    """An empty batch leaves gradients of zero."""
    x, w = parts(0, 9).requires_grad_(), parts(7, 9).requires_grad_()
    b = parts(7).requires_grad_() if bias else None
    y = lm.mx_linear(x, w, b)
    assert y.shape == (0, 7)
    dx, dw, *db = torch.autograd.grad(y.sum(), [t for t in (x, w, b) if t is not None])
    assert dx.shape == (0, 9) and dw.shape == (7, 9) and dw.dtype == w.dtype and not dw.any()
    assert all(d.shape == (7,) and not d.any() for d in db)


def test_derivatives_of_gradients_raise(calls):
    """The backward passes have no derivative of their own.  A gradient that is used as a number is
    as before; a derivative that reaches it, by whatever way, raises and does not leave it out."""
    x, w = parts(4, 9, seed=1).requires_grad_(), parts(7, 9, seed=2).requires_grad_()
    v = parts(7, seed=3).requires_grad_()
    for loss in (lambda y: y.sum(), lambda y: y.square().sum(), lambda y: (y * v).sum()):
        dx, dw = torch.autograd.grad(loss(lm.mx_linear(x, w)), (x, w), create_graph=True)
        want = torch.autograd.grad(loss(x @ w.T), (x, w))
        assert torch.allclose(dx, want[0], atol=1e-5) and torch.allclose(dw, want[1], atol=1e-5)
        for of, to in ((dx, w), (dw, x), (dx, x)):
            with pytest.raises(RuntimeError, match="differentiable once"):
                torch.autograd.grad(of.square().sum() + to.sum(), to, retain_graph=True)
    z, ids, lps = parts(4, 33).requires_grad_(), torch.arange(12, dtype=torch.int32).view(4, 3), parts(4, 3)
    dz, = torch.autograd.grad(lm.distill(z, ids, lps).sum(), z, create_graph=True)
    assert torch.allclose(dz, torch.autograd.grad(plain_distill(z, ids, lps, 1.0).sum(), z)[0], atol=1e-5)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(dz.square().sum() + z.sum(), z)


def test_derivative_through_the_incoming_gradient_raises(calls):
    """v weighs the outputs, so the gradient of x depends on it through what arrives."""
    x, w, v = parts(4, 9).requires_grad_(), parts(7, 9).requires_grad_(), parts(7).requires_grad_()
    dx, = torch.autograd.grad((lm.mx_linear(x, w) * v).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(dx.square().sum() + v.sum(), v)


def test_gradients_hold_none_of_the_activations(calls):
    """Between the passes a layer keeps its packed operands, not its input."""
    import weakref
    w = parts(7, 9, seed=2).requires_grad_()
    x = parts(4, 9, seed=1) * 2
    alive = weakref.ref(x)
    y = lm.mx_linear(x, w)
    del x
    assert alive() is None
    y.sum().backward()
    assert w.grad.shape == w.shape


def test_a_context_of_ones_own(calls):
    """Work on two streams at once needs a context for each: the one that is given serves every call
    of the forward and of the backward pass."""
    mine = object()
    x, w = parts(4, 9).requires_grad_(), parts(7, 9).requires_grad_()
    lm.mx_linear(x, w, ctx=mine).sum().backward()
    z = parts(4, 33).requires_grad_()
    lm.distill(z, torch.arange(12, dtype=torch.int32).view(4, 3), parts(4, 3), ctx=mine).sum().backward()
    assert len(calls) == 8 and all(kw["ctx"] is mine for _, kw in calls)
    del calls[:]
    lm.mx_linear(x, w).sum().backward()
    assert len(calls) == 6 and all(kw["ctx"] is None for _, kw in calls)
