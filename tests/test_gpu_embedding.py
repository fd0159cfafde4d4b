"""Token embeddings and their gradient, through the library, against the 64-bit definitions."""
import numpy as np
import pytest
import torch

from oracle import layers
from tests.gpu_helpers import gq, host, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def code(g, dtype):
    return g.BF16 if dtype == BF16 else g.F32


def make(rows, cols, dtype, seed):
    return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def some_ids(tokens, vocab, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, vocab, tokens)
    if kind == "mixed":
        hot = rng.random(tokens)
        ids[hot < 0.3] = vocab // 2
        ids[hot > 0.95] = rng.choice([-1, vocab, -5, 2 ** 40, vocab + 7], tokens)[hot > 0.95]
    elif kind == "one":
        ids[:] = vocab - 1
    elif kind == "none":
        ids[:] = -1
    return torch.from_numpy(ids)


@pytest.mark.parametrize("tokens,vocab,dim", [(1, 1, 1), (5, 3, 7), (33, 100, 8), (70, 1000, 130), (9, 50, 1029), (300, 20, 2056)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("scale", [1.0, 0.3])
def test_lookup(tokens, vocab, dim, dtype, out, scale):
    """One rounding of fp32, and for bf16 one more: half a step of each; a scale of 1 is exact where the
    output holds the table's type."""
    say("embedding", tokens, vocab, dim, dtype, out, scale)
    g = gq()
    table, ids = make(vocab, dim, dtype, dim), some_ids(tokens, vocab, tokens)
    got = g.embedding(table, ids.cuda(), scale=scale, out_dtype=code(g, out))
    assert got.dtype == out
    want = layers.embedding(table.double().cpu().numpy(), ids.numpy(), scale)
    eps = 2.0 ** -24 + (2.0 ** -8 if out == BF16 else 0)
    if scale == 1.0 and not (dtype == F32 and out == BF16):
        eps = 0
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= np.abs(want) * eps * (1 + 2.0 ** -7))


def test_lookup_far_into_a_table():
    """Offsets beyond 2^32 bytes and beyond 2^31 elements."""
    say("embedding of a large table")
    g = gq()
    vocab, dim = 300000, 8192
    table = torch.zeros(vocab, dim, dtype=BF16, device="cuda")
    ids = torch.tensor([0, 262143, 262144, 299999, 131072, 150000], device="cuda")
    table[ids] = make(6, dim, BF16, 1)
    assert torch.equal(g.embedding(table, ids), table[ids])
    grad = torch.empty(vocab, dim, dtype=BF16, device="cuda").fill_(1)
    d = make(6, dim, BF16, 2)
    g.embedding_grad(d, ids, vocab, out=grad, out_dtype=g.BF16)
    assert torch.equal(grad[ids], d)
    rows = grad.view(torch.int32).any(1).nonzero().flatten()
    assert rows.tolist() == sorted(ids.tolist())


def check_gradient(got, dout, ids, vocab, scale, old=None):
    """A sum of c terms in fp32 in any order, its product with the scale, the old value and the output's
    type: (c + 1) 2^-24 of the magnitudes' sum, one rounding of the total, half a step of bf16."""
    want, mass, count = layers.embedding_grad(dout.double().cpu().numpy(), ids.numpy(), vocab, scale)
    bound = mass * (count[:, None] + 1) * 2.0 ** -24
    if old is not None:
        want = want + old
        bound = bound + np.abs(want) * 2.0 ** -24
    if got.dtype == BF16:
        bound = bound * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8
    d = np.abs(got.double().cpu().numpy() - want)
    assert np.all(d <= bound * (1 + 1e-5)), (d - bound).max()
    return count


CASES = [(1, 1, 1, "mixed"), (3, 7, 5, "mixed"), (64, 10, 33, "one"), (65, 10, 33, "one"), (128, 4, 40, "one"), (129, 300, 96, "one"),
         (300, 5, 64, "mixed"), (1000, 1000, 40, "mixed"), (1025, 257, 8, "even"), (2500, 30, 520, "mixed"), (777, 3000, 1, "mixed"),
         (4100, 9, 100, "even"), (40, 20, 16, "none"), (5000, 1, 12, "mixed"), (70000, 400, 4, "mixed"), (1500, 250000, 8, "even")]


@pytest.mark.parametrize("tokens,vocab,dim,kind", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("out", [F32, BF16])
def test_gradient(tokens, vocab, dim, kind, dtype, out):
    say("embedding gradient", tokens, vocab, dim, kind, dtype, out)
    g = gq()
    dout, ids = make(tokens, dim, dtype, tokens), some_ids(tokens, vocab, tokens + dim, kind)
    buf = torch.full((vocab, dim), 9.0, dtype=out, device="cuda")
    got = g.embedding_grad(dout, ids.cuda(), vocab, scale=1.25, out=buf, out_dtype=code(g, out))
    check_gradient(got, dout, ids, vocab, 1.25)
    again = g.embedding_grad(dout, ids.cuda(), vocab, scale=1.25, out_dtype=code(g, out))
    assert torch.equal(again, got)


@pytest.mark.parametrize("tokens,vocab,dim,kind", [(50, 30, 17, "mixed"), (3000, 40, 130, "mixed"), (200, 5000, 64, "even"), (5, 4, 8, "none")])
@pytest.mark.parametrize("out", [F32, BF16])
def test_gradient_added(tokens, vocab, dim, kind, out):
    """Rows of no token are not touched, whatever they hold."""
    say("embedding gradient added", tokens, vocab, dim, kind, out)
    g = gq()
    dout, ids = make(tokens, dim, BF16, 4), some_ids(tokens, vocab, 5, kind)
    buf = make(vocab, dim, out, 6)
    old = buf.double().cpu().numpy()
    free = np.setdiff1d(np.arange(vocab), ids.numpy())
    got = g.embedding_grad(dout, ids.cuda(), vocab, scale=0.5, out=buf, out_dtype=code(g, out), accumulate=True)
    assert got is buf
    check_gradient(got, dout, ids, vocab, 0.5, old)
    assert np.array_equal(got.double().cpu().numpy()[free], old[free])
    buf[torch.from_numpy(free).cuda()] = float("nan")
    g.embedding_grad(dout, ids.cuda(), vocab, out=buf, out_dtype=code(g, out), accumulate=True)
    nan = torch.isnan(buf).all(1).cpu().numpy()
    assert np.array_equal(np.flatnonzero(nan), free)


def test_order_is_the_tokens():
    """fp32 sums of few tokens are taken in the tokens' order: equal to adding them one after another."""
    say("embedding gradient order")
    g = gq()
    tokens, vocab, dim = 3000, 100, 24
    dout, ids = make(tokens, dim, F32, 1), some_ids(tokens, vocab, 2, "even")
    got = host(g.embedding_grad(dout, ids.cuda(), vocab))
    d = host(dout)
    for v in range(vocab):
        at = np.flatnonzero(ids.numpy() == v)
        assert len(at) <= 64
        s = np.zeros(dim, np.float32)
        for t in at:
            s = s + d[t]
        assert np.array_equal(got[v], s)


def test_values_without_numbers():
    """Infinities and NaN of padding tokens stay out; a real token's reach its row alone."""
    say("embedding values")
    g = gq()
    table = make(6, 20, F32, 1)
    table[2, 3] = float("nan")
    ids = torch.tensor([-1, 2, 0, 6, 2], device="cuda")
    got = g.embedding(table, ids)
    assert torch.isnan(got).nonzero().tolist() == [[1, 3], [4, 3]] and not got[0].any() and not got[3].any()
    d = torch.ones(5, 20, device="cuda")
    d[0] = float("inf")
    d[3] = float("nan")
    d[2, 7] = float("-inf")
    grad = g.embedding_grad(d, ids, 6)
    assert torch.isinf(grad).nonzero().tolist() == [[0, 7]] and not torch.isnan(grad).any() and torch.all(grad[2] == 2)


def test_strides():
    """Rows of wider matrices, at any element's alignment; what lies between the rows stays."""
    say("embedding strides")
    g = gq()
    for dtype in (F32, BF16):
        wide = make(40, 101, dtype, 3)
        ids = some_ids(90, 40, 4)
        out = torch.full((93, 77), 5.0, dtype=dtype, device="cuda")
        got = g.embedding(wide[:, :67], ids.cuda(), out=out[:90, :67])
        want = layers.embedding(wide[:, :67].double().cpu().numpy(), ids.numpy(), 1.0)
        assert np.array_equal(got.double().cpu().numpy(), want)
        assert torch.all(out[90:] == 5) and torch.all(out[:, 67:] == 5)
        dout = make(90, 75, dtype, 5)
        grad = torch.full((42, 70), 5.0, dtype=F32, device="cuda")
        check_gradient(g.embedding_grad(dout[:, :67], ids.cuda(), 40, out=grad[:40, :67]), dout[:, :67], ids, 40, 1.0)
        assert torch.all(grad[40:] == 5) and torch.all(grad[:, 67:] == 5)


def test_by_differences():
    """The gradient of sum(w * embedding) in one direction of the table."""
    say("embedding gradient by differences")
    g = gq()
    table, ids, w = make(30, 16, F32, 1), some_ids(200, 30, 2).cuda(), make(200, 16, F32, 3)
    d = make(30, 16, F32, 4)
    grad = g.embedding_grad(w, ids, 30, scale=2.0)

    def f(t):
        return (g.embedding(t, ids, scale=2.0).double() * w.double()).sum()

    slope = (f(table + 0.5 * d) - f(table - 0.5 * d)).item()     # the function is linear
    want = (grad.double() * d.double()).sum().item()
    # 3200 products of fp32 values, each off by 2^-24 of some 10, and the sums' roundings
    assert abs(slope - want) <= 3200 * 10 * 2.0 ** -23 * 4


def test_empty_and_refused():
    say("embedding refusals")
    g = gq()
    table, none = make(4, 8, F32, 1), torch.zeros(0, dtype=torch.int64, device="cuda")
    assert g.embedding(table, none).shape == (0, 8)
    assert not g.embedding_grad(torch.zeros(0, 8, device="cuda"), none, 4).any()
    assert torch.equal(g.embedding(table[:0], torch.zeros(3, dtype=torch.int64, device="cuda")), torch.zeros(3, 8, device="cuda"))
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    d = torch.zeros(3, 8, device="cuda")
    assert g.embedding_grad(d, ids, 0).shape == (0, 8)
    for call in (lambda: g.embedding(table, ids.int()), lambda: g.embedding(table.half(), ids), lambda: g.embedding(table.cpu(), ids),
                 lambda: g.embedding(table, ids, out=torch.zeros(3, 8, device="cuda"), out_dtype=g.BF16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: g.embedding(table, ids.view(1, 3)), lambda: g.embedding(table, ids, out=torch.zeros(2, 8, device="cuda")),
                 lambda: g.embedding(table.T, ids), lambda: g.embedding_grad(d, ids[:2], 4), lambda: g.embedding_grad(d, ids, 4, accumulate=True),
                 lambda: g.embedding_grad(d, ids, 4, out=torch.zeros(4, 7, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    flat = torch.zeros(64, device="cuda")
    for call in (lambda: g.embedding(flat[1:33].view(4, 8), ids), lambda: g.embedding(table[:3], ids, out=table[:3]),
                 lambda: g.embedding_grad(d, ids, 3, out=d)):
        with pytest.raises(g.GQError):
            call()
