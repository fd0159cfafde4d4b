"""The autograd functions on tensors that begin at any element: the same bits as from whole copies."""
import pytest
import torch

from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu


def parts(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_outputs_joined(dtype):
    from allreduce_compatible_gradient_amd import lm
    say("lm cat", dtype)
    g = gq()
    w = parts(7, 45, seed=1).requires_grad_()
    x = [parts(n, 45, seed=n, dtype=dtype).requires_grad_() for n in (5, 6)]
    weight = parts(11, 7, seed=4, dtype=dtype)
    got = torch.autograd.grad((torch.cat([lm.mx_linear(t, w, seed=9) for t in x]) * weight).sum(), [w] + x)
    each = [torch.autograd.grad(lm.mx_linear(t, w, seed=9), (t, w), d.clone()) for t, d in zip(x, weight.split([5, 6]))]
    assert torch.equal(got[1], each[0][0]) and torch.equal(got[2], each[1][0])
    assert torch.equal(got[0], each[0][1] + each[1][1])
    z = [parts(n, 333, seed=n, dtype=dtype).requires_grad_() for n in (5, 7)]
    teacher = [g.token_logprobs(parts(n, 333, seed=20 + n), torch.zeros(n, dtype=torch.int64, device="cuda"), 9)[2:]
               for n in (5, 7)]
    weight = parts(12, seed=8)
    got = torch.autograd.grad((torch.cat([lm.distill(t, *a, tail=True) for t, a in zip(z, teacher)]) * weight).sum(), z)
    for d, t, a, v in zip(got, z, teacher, weight.split([5, 7])):
        assert torch.equal(d, g.distill_loss(t.detach(), *a, tail=True, row_weight=v.clone())[1])


def test_views():
    from allreduce_compatible_gradient_amd import lm
    say("lm views")
    flat = parts(1 + 63 + 7, seed=1)
    w, b = flat[1:64].view(7, 9), flat[64:]
    for x in (parts(6, 9, seed=3)[1:], parts(9, 12, seed=2).T, parts(6, 13, seed=4)[:, 2:11]):
        assert torch.equal(lm.mx_linear(x, w, b), lm.mx_linear(x.clone(memory_format=torch.contiguous_format), w.clone(), b.clone()))
    z, ids, lps = parts(6, 333, seed=6), torch.arange(30, dtype=torch.int32, device="cuda").view(6, 5), parts(6, 5, seed=7)
    assert torch.equal(lm.distill(z[1:], ids[1:], lps[1:]), lm.distill(z, ids, lps)[1:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_tokens(dtype):
    from allreduce_compatible_gradient_amd import lm
    say("lm no tokens", dtype)
    x, w, b = (parts(*s, dtype=d).requires_grad_() for s, d in (((0, 45), dtype), ((7, 45), torch.float32), ((7,), torch.float32)))
    y = lm.mx_linear(x, w, b)
    assert y.shape == (0, 7) and y.dtype == dtype
    dx, dw, db = torch.autograd.grad(y.sum(), (x, w, b))
    assert dx.shape == x.shape and dw.shape == w.shape and not dw.any() and not db.any()
    z = parts(0, 333, dtype=dtype).requires_grad_()
    loss = lm.distill(z, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), torch.zeros(0, 3, device="cuda"), tail=True)
    assert loss.shape == (0,) and torch.autograd.grad(loss.sum(), z)[0].shape == z.shape


def test_two_streams_with_a_context_each():
    """Layers whose products are split along K (their partial products lie in the context's scratch
    memory) and distillation in slices, on two streams at once: the bits of one after the other."""
    from allreduce_compatible_gradient_amd import lm
    say("lm two streams")
    g = gq()
    teacher = [g.token_logprobs(parts(3, 9001, seed=s), torch.zeros(3, dtype=torch.int64, device="cuda"), 9)[2:] for s in (1, 2)]
    x = [parts(40, 9000, seed=10 + s, dtype=torch.bfloat16) for s in (1, 2)]
    z = [parts(3, 9001, seed=20 + s) for s in (1, 2)]
    w = parts(300, 9000, seed=30)

    def both(i, ctx):
        a, b, c = x[i].detach().requires_grad_(), w.detach().requires_grad_(), z[i].detach().requires_grad_()
        y = lm.mx_linear(a, b, seed=i, ctx=ctx)
        loss = lm.distill(c, *teacher[i], tail=True, ctx=ctx)
        return [y, loss, *torch.autograd.grad((y.float().square().sum() + loss.sum()), (a, b, c))]

    ctxs = [g.Context(), g.Context()]
    want = [both(i, ctxs[i]) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [None, None]
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = both(i, ctxs[i])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
