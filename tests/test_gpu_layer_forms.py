"""Every form that a rule on sizes chooses for the operators around a model's layers: the tiles of updates
and of 8-bit products with every epilogue, tall matrices, the sort's forms, and rows quantised on the way
into a product with more steps than a wave has on their way together."""
import math

import numpy as np
import pytest
import torch

from oracle import layers
from tests import layer_forms
from tests.gpu_helpers import dev, gq, host, say
from tests.test_gpu_embedding import check_gradient, make, some_ids
from tests.test_gpu_int8 import packed, product_case, values

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ----------------------------------------------------------------------------- updates
def halves(x, scale):
    return (x * scale).half().double() / scale


def definition(g, rounded, steps=5):
    """The update of a matrix in 64 bits; or with the roundings of layers.orthogonalise_in_halves' larger
    form, at the same places."""
    a, b, c = layers.QUINTIC
    flip = g.shape[0] > g.shape[1]
    x = g.double().T.contiguous() if flip else g.double()
    x = x / torch.linalg.matrix_norm(x)
    if rounded:
        x = x.float().double()
    for step in range(steps):
        if not rounded:
            p = x @ x.T.contiguous()
            x = a * x + (b * p + c * (p @ p)) @ x
            continue
        h = halves(x, 256.0)
        p = (h @ h.T.contiguous()).float().double()
        d = p.diagonal().clone()
        f = halves(p - torch.diag(d), 1024.0)
        sq = f @ f
        q = b * f + c * ((d[:, None] + d) * f + sq)
        diag = b * d + c * (d * d + sq.diagonal())
        q.fill_diagonal_(0.0)
        x = (a * x + diag[:, None] * (h if step < steps - 2 else x) + halves(q, 1024.0) @ h).float().double()
    if rounded:
        x = x.float().bfloat16().double()
    return x.T if flip else x


@pytest.mark.parametrize("batch,n,m", list(layer_forms.UPDATES))
@pytest.mark.parametrize("tall", [False, True])
def test_update(batch, n, m, tall):
    """As far from the definition as the same roundings take it, by their law: norms of 4000 roundings and
    more differ by a few percent, a quarter is allowed, and 2^-14 for the fp32 sums; an element by half
    a bf16's step and ten times the roundings' root mean square.  Rows of wider matrices, whose rest stays."""
    say("update's form", batch, n, m, tall)
    rows, cols = (m, n) if tall else (n, m)
    gen = torch.Generator("cuda").manual_seed(n + m)
    g = torch.randn(batch, rows, cols, device="cuda", generator=gen)
    g += 3 * torch.randn(batch, rows, 1, device="cuda", generator=gen) * torch.randn(batch, 1, cols, device="cuda", generator=gen)
    wide = torch.full((batch, rows + 1, cols + 3), 3.0, dtype=BF16, device="cuda")
    got = gq().orthogonalise(g, out=wide[:, :rows, :cols])
    assert bool((wide[:, rows:] == 3).all()) and bool((wide[:, :, cols:] == 3).all())
    for i in sorted({0, 1, batch // 2, batch - 1} & set(range(batch))):
        want = definition(g[i], False)
        own, norm = (definition(g[i], True) - want).norm().item(), want.norm().item()
        d = got[i].double() - want
        assert d.norm().item() <= 1.25 * own + 2.0 ** -14 * norm, (i, d.norm().item() / norm, own / norm)
        rms = own / math.sqrt(rows * cols)
        assert bool((d.abs() <= want.abs() * 2.0 ** -8 + 10 * rms).all()), i
    assert torch.equal(gq().orthogonalise(g), got)


# ----------------------------------------------------------------------------- products
@pytest.mark.parametrize("m,n,k", list(layer_forms.PRODUCTS))
@pytest.mark.parametrize("form", ["plain", "bias", "accumulate", "both"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product(m, n, k, form, dtype):
    """Exact sums (64 bits hold them); three roundings of the product, one more of each sum, half a step
    of the type.  Rows as they come, and rows of a wider matrix at any element, whose rest stays."""
    say("product's form", m, n, k, form, dtype)
    g = gq()
    gen = torch.Generator("cuda").manual_seed(m + n + k)
    pitch = g.int_pitch(k)

    def matrix(rows):
        codes = torch.zeros(rows, pitch, dtype=torch.int8, device="cuda")
        codes[:, :k] = torch.randint(-127, 128, (rows, k), device="cuda", generator=gen).to(torch.int8)
        return g.IntTensor(codes, torch.rand(rows, device="cuda", generator=gen) * 0.01 + 1e-3, k)

    a, b = matrix(m), matrix(n)
    bias = torch.randn(n, device="cuda", generator=gen) if form in ("bias", "both") else None
    old = torch.randn(m, n, device="cuda", generator=gen).to(dtype) if form in ("accumulate", "both") else None
    product = (a.codes.double() @ b.codes.double().T) * a.scales.double()[:, None] * b.scales.double()
    want, bound = product, 3 * product.abs() * 2.0 ** -24
    if bias is not None:
        want = want + bias.double()
        bound = bound + want.abs() * 2.0 ** -24
    if old is not None:
        want = want + old.double()
        bound = bound + want.abs() * 2.0 ** -24
    if dtype == BF16:
        bound = bound * (1 + 2.0 ** -8) + want.abs() * 2.0 ** -8
    del product
    for more in (0, 5):
        wide = torch.full((m + 1, n + more), 7.0, dtype=dtype, device="cuda")
        out = wide[:m, :n]
        if old is not None:
            out.copy_(old)
        g.int_matmul(a, b, bias=bias, out_dtype=g.BF16 if dtype == BF16 else g.F32, out=out, accumulate=old is not None)
        assert bool(((out.double() - want).abs() <= bound * (1 + 1e-6)).all()), more
        assert bool((wide[m:] == 7).all()) and bool((wide[:, n:] == 7).all()), more


@pytest.mark.parametrize("m,k", [(1, 11008), (1, 20001), (2, 8193), (2, 11008), (3, 10000), (4, 5001), (7, 4224), (1, 32768), (16, 2048),
                                 # rows that a launch of their own packs
                                 (1, 32769), (4, 11008), (9, 4096), (16, 11008)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_rows_quantised_on_the_way(m, k, dtype):
    """The bits of the packed rows, and those of the definition within three roundings."""
    say("few rows quantised", m, k, dtype)
    g = gq()
    n = 45
    _, _, b, sb, bias = product_case(1, n, k, 8)
    x = values(m, k, 9, dtype).cuda()
    q, _ = g.int_quantize(x)
    w = packed(g, b, sb, k)
    for out in (g.F32, g.BF16):
        assert torch.equal(g.int_matmul(x, w, out_dtype=out, bias=dev(bias)), g.int_matmul(q, w, out_dtype=out, bias=dev(bias)))
    codes, scales = layers.quantize(x.float().cpu().numpy(), 0)
    want, mag = layers.matmul(codes, scales, b, sb)
    assert np.all(np.abs(host(g.int_matmul(x, w, out_dtype=g.F32)) - want) <= 3 * mag * 2.0 ** -24 * (1 + 1e-6) + 1e-44)


# ----------------------------------------------------------------------------- the gradient's sort
@pytest.mark.parametrize("tokens", [1024, 2047, 2048, 2049, 8192, 8193, 12001, 16384, 16385, 40000])
@pytest.mark.parametrize("vocab,kind", [(700, "mixed"), (50257, "mixed"), (300000, "even")])
def test_gradient_of_many_tokens(tokens, vocab, kind):
    """Each number of tokens that a wave holds at its limits, and one id of a third of them."""
    say("embedding gradient", tokens, vocab, kind)
    g = gq()
    dim = 5
    dout, ids = make(tokens, dim, BF16, tokens), some_ids(tokens, vocab, tokens + vocab, kind)
    got = g.embedding_grad(dout, ids.cuda(), vocab)
    check_gradient(got, dout, ids, vocab, 1.0)
    assert torch.equal(g.embedding_grad(dout, ids.cuda(), vocab), got)
