"""What the linear layers ask the library for, with and without a gradient to come: on a stand-in for the
binding that records its calls (CPU only)."""
import pytest
import torch

from allreduce_compatible_gradient_amd import gq, lm

CALLS = {"int": ("int_quantize", "int_matmul", lm.int_linear), "mx": ("mx_quantize", "mx_matmul", lm.mx_linear)}


@pytest.fixture
def made(monkeypatch):
    calls = []

    def quantize(x, rounding=0, seed=0, worker=0, index_base=0, by_rows=True, by_cols=False, **kw):
        calls.append((tuple(x.shape), by_rows, by_cols))
        return tuple(x.shape), tuple(x.shape)[::-1] if by_cols else None

    def matmul(a, b, bias=None, out_dtype=gq.BF16, **kw):
        assert a[1] == b[1]
        return torch.zeros(1, 1, dtype=torch.float32 if out_dtype == gq.F32 else torch.bfloat16).expand(a[0], b[0])

    for q, m, _ in CALLS.values():
        monkeypatch.setattr(gq, q, quantize)
        monkeypatch.setattr(gq, m, matmul)
    return calls


def leaf(*shape, grad=False):
    return torch.zeros(1, 1).expand(*shape).requires_grad_(grad)


@pytest.mark.parametrize("kind", list(CALLS))
@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_without_gradients_nothing_is_packed_by_columns(made, kind, off):
    linear = CALLS[kind][2]
    x, w, b = leaf(6, 3), leaf(5, 3, grad=True), torch.zeros(5, requires_grad=True)
    with off():
        y = linear(x, w, b)
    assert y.shape == (6, 5) and not y.requires_grad
    assert made == [((6, 3), True, False), ((5, 3), True, False)]
    made.clear()
    linear(x, w, b)         # the weights' gradient needs the inputs by columns
    assert made == [((6, 3), True, True), ((5, 3), True, False)]
    made.clear()
    linear(leaf(6, 3, grad=True), w.detach())
    assert made == [((6, 3), True, False), ((5, 3), True, True)]


def test_more_outputs_than_the_draws_of_a_backward_pass(made):
    """The gradient's rounding has 2^32 draws: a layer of more outputs is refused before its forward
    work, unless no gradient is wanted."""
    x, w = leaf(98304, 1), leaf(50257, 1)
    for a, c in ((leaf(98304, 1, grad=True), w), (x, leaf(50257, 1, grad=True))):
        with pytest.raises(ValueError, match="2\\^32"):
            lm.int_linear(a, c)
    assert made == []
    assert lm.int_linear(x, w).shape == (98304, 50257)
    with torch.no_grad():
        assert lm.int_linear(x, leaf(50257, 1, grad=True)).shape == (98304, 50257)
    # a bias alone has a gradient without draws; 2^32 entries are within the limit
    assert lm.int_linear(x, w, torch.zeros(50257, requires_grad=True)).requires_grad
    assert lm.int_linear(leaf(65536, 1), leaf(65536, 1, grad=True)).shape == (65536, 65536)
