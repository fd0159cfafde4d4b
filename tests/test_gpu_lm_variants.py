"""Every size that the language-model operators' rules treat apart: rows held by 256 threads with 8
and 26 chunks each and by 512 with 8 and 16, and the product's 256 x 256 tiles with odd and even
numbers of K steps, rows on and off 128-byte lines, bias, old values and K splits."""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu


def bits(t):
    t = torch.where(torch.isnan(t), torch.full_like(t, float("nan")), t)
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def teacher(z, top, temperature, rng):
    t = torch.log_softmax((z.double() + 1.0 * torch.from_numpy(rng.standard_normal(z.shape))) / temperature, 1)
    v, i = t.topk(top, 1)
    return i.to(torch.int32).numpy(), v.float().numpy()


# (dtype, vocab): the last row length of a form, the first of the next, and the middle of each
HELD = [(torch.bfloat16, v) for v in (16320, 16321, 20011, 32704, 32705, 40009, 50257, 53184, 53185, 60013, 65472)] + \
       [(torch.float32, v) for v in (16320, 16321, 20011, 32704)]


@pytest.mark.parametrize("dtype,vocab", HELD)
@pytest.mark.parametrize("tail", [False, True])
def test_held_rows(dtype, vocab, tail):
    """130 rows are one slice each.  Padding, repeats, masks, a NaN, taught entries at a row's ends;
    the gradient fused, apart and in place has the same bits, and strided rows too.  Tolerances: a
    thread's share of the row and the joins in the logarithms, then a rounding."""
    say("held rows", dtype, vocab, tail)
    g = gq()
    rows, top, temperature = 130, 24, 1.25
    rng = np.random.default_rng(vocab)
    z = torch.from_numpy(rng.standard_normal((rows, vocab)).astype(np.float32) * 3).to(dtype)
    some = list(range(9)) + [100, 129]
    ids, lps = np.empty((rows, top), np.int32), np.empty((rows, top), np.float32)
    for r in range(0, rows, 32):
        ids[r:r + 32], lps[r:r + 32] = teacher(z[r:r + 32].float(), top, temperature, rng)
    ids[0] = -1                                     # taught nothing
    ids[1, 5:] = -1
    ids[2, 3], ids[2, 7] = ids[2, 0], vocab         # occurs again; outside
    ids[3, :4] = [0, 1, vocab - 1, vocab - 2]
    z[4, 64:vocab - 64] = float("-inf")
    ids[4, :2] = [0, vocab - 1]
    z[5, vocab // 2] = float("nan")
    z[6, :8] = float("-inf")
    ids[7] = (np.arange(top) + 8 * (vocab // 8) - 16) % vocab
    w = rng.random(rows).astype(np.float32) + 0.1
    zd, wd = z.cuda(), torch.from_numpy(w).cuda()
    args = (torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda(), temperature, tail)
    loss, grad = g.distill_loss(zd, *args, row_weight=wd)
    alone, stats = g.distill_loss(zd, *args)
    apart = g.distill_grad(zd, *args, stats, wd)
    assert torch.equal(bits(alone), bits(loss)) and torch.equal(bits(apart), bits(grad))
    wide = torch.full((rows, vocab + 5), 3.0, dtype=dtype, device="cuda")
    view = wide[:, :vocab]
    view.copy_(zd)
    strided, _ = g.distill_loss(view, *args, row_weight=wd, dlogits=view)
    assert bool((wide[:, vocab:] == 3).all())
    # other places in their lines: the same chunks in another order, so not the same bits
    place = zd.clone()
    g.distill_loss(place, *args, row_weight=wd, dlogits=place)
    assert torch.equal(bits(place), bits(grad))
    del wide, apart, place
    rl, rg, _ = lm.distill(z[some].float().numpy(), ids[some], lps[some], temperature, tail, w[some])
    eps = (vocab / 256 + 64) * 2.0 ** -22
    for got in (loss, strided):
        got = got[some].double().cpu().numpy()
        with np.errstate(all="ignore"):
            tol = 6 * temperature ** 2 * eps + np.abs(rl) * 2.0 ** -22
            assert np.all((got == rl) | (np.isnan(got) & np.isnan(rl)) | (np.abs(got - rl) <= tol)), (got, rl)
    got = grad[some].double().cpu().numpy()
    q = np.exp(lm.log_softmax(z[some].float().numpy(), temperature))
    scale = (w[some] * temperature)[:, None].astype(np.float64)
    with np.errstate(all="ignore"):
        tol = 4 * eps * (np.abs(rg) + scale * q) + 2.0 ** -125
        if dtype == torch.bfloat16:
            tol = tol + np.abs(rg) * 2.0 ** -8
        bad = ~((got == rg) | (np.isnan(got) & np.isnan(rg)) | (np.abs(got - rg) <= tol))
    bad[5] = False                                  # the row with a NaN: below
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], rg[bad][:4])
    assert np.isnan(got[5]).all() and float(loss[0]) == 0 and not got[0].any()


@pytest.mark.parametrize("rows,vocab", [(9, 700), (9, 9001), (1030, 70001), (9, 140001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tail", [False, True])
def test_fused_apart_and_in_place_agree_on_odd_rows(rows, vocab, dtype, tail):
    """Held rows, slices, and rows of one slice that are not held: every bit, infinities and NaN
    included, is the same whichever way the gradient is asked for."""
    say("same bits", rows, vocab, dtype, tail)
    g = gq()
    gen = torch.Generator("cuda").manual_seed(vocab)
    z = torch.empty(rows, vocab, device="cuda", dtype=dtype).normal_(generator=gen)
    ids = (torch.arange(rows * 6, dtype=torch.int32, device="cuda").view(rows, 6) * 37) % vocab
    lps = torch.log_softmax(torch.empty(rows, 7, device="cuda").normal_(generator=gen), 1)[:, :6].contiguous()
    z[0] = float("-inf")
    z[1, 5] = float("nan")
    z[2, 6] = float("inf")
    ids[3] = -1
    z[4] = float("-inf")
    z[4, ids[4].long()] = 1.0
    z[5] = torch.finfo(dtype).min
    z[6, ids[6, 0].long()] = float("-inf")
    lps[7] = -200.0
    z[8, ids[8].long()] = 300.0
    w = torch.rand(rows, device="cuda", generator=gen)
    w[7] = 0.0
    args = (ids, lps, 1.0, tail)
    loss, grad = g.distill_loss(z, *args, row_weight=w)
    alone, stats = g.distill_loss(z, *args)
    assert torch.equal(bits(alone), bits(loss))
    assert torch.equal(bits(g.distill_grad(z, *args, stats, w)), bits(grad))
    place = z.clone()
    g.distill_loss(place, *args, row_weight=w, dlogits=place)
    assert torch.equal(bits(place), bits(grad))
    assert bool(torch.isnan(loss[1:3]).all()) and float(loss[3]) == 0 and not bool(grad[3].any())
    assert bool(torch.isfinite(loss[7:9]).all()) and bool(torch.isfinite(grad[7:].float()).all())


@pytest.mark.parametrize("m,n,k", [(2300, 4096, 256), (2300, 4099, 700), (2309, 4096, 1280), (2200, 4096, 1500)])
@pytest.mark.parametrize("out_dtype", [0, 1])
def test_large_tiles(m, n, k, out_dtype):
    """9 or 10 x 16 or 17 tiles of 256 x 256 with 1, 3, 5 and 6 steps of K, ragged in M; n = 4096 puts
    the rows on lines and 4099 off them.  Plain, with a bias, added to old values, and both."""
    say("large tiles", m, n, k, out_dtype)
    g = gq()
    gen = torch.Generator("cuda").manual_seed(m + n + k)
    qa, _ = g.mx_quantize(torch.randn(m, k, device="cuda", generator=gen))
    qb, _ = g.mx_quantize(torch.randn(n, k, device="cuda", generator=gen) * 0.1)
    va, vb = g.mx_dequantize(qa, g.F32).double(), g.mx_dequantize(qb, g.F32).double()
    ref = va @ vb.T
    bound = (va.abs() @ vb.abs().T) * (k / 64 + 64) * 2.0 ** -24
    bias = torch.randn(n, device="cuda", generator=gen)
    old = torch.randn(m, n + 3, device="cuda", generator=gen).to(torch.float32 if out_dtype == 0 else torch.bfloat16)
    for b in (None, bias):
        for add in (False, True):
            for wide in (False, True):
                buf = old.clone() if wide else old[:, :n].contiguous()
                out = buf[:, :n]
                g.mx_matmul(qa, qb, bias=b, out_dtype=out_dtype, out=out, accumulate=add)
                more = [t for t in (None if b is None else b.double(), old[:, :n].double() if add else None)
                        if t is not None]
                want, tol = ref.clone(), bound.clone()
                for t in more:
                    want += t
                    tol += (ref.abs() + t.abs()) * 2.0 ** -22
                if out_dtype == 1:
                    tol += want.abs() * 2.0 ** -8
                assert bool(((out.double() - want).abs() <= tol).all()), (b is not None, add, wide)
                assert torch.equal(buf[:, n:], old[:, n:] if wide else old[:, :0])


@pytest.mark.parametrize("m,n,k", [(40, 300, 9000), (100, 90, 40000), (64, 200, 6300)])
@pytest.mark.parametrize("out_dtype", [0, 1])
def test_splits_with_bias_and_old_values(m, n, k, out_dtype):
    say("splits epilogue", m, n, k, out_dtype)
    g = gq()
    gen = torch.Generator("cuda").manual_seed(k)
    qa, _ = g.mx_quantize(torch.randn(m, k, device="cuda", generator=gen))
    qb, _ = g.mx_quantize(torch.randn(n, k, device="cuda", generator=gen) * 0.1)
    bias = torch.randn(n, device="cuda", generator=gen)
    plain = g.mx_matmul(qa, qb, out_dtype=g.F32).double()
    old = torch.randn(m, n + 3, device="cuda", generator=gen).to(torch.float32 if out_dtype == 0 else torch.bfloat16)
    buf = old.clone()
    g.mx_matmul(qa, qb, bias=bias, out_dtype=out_dtype, out=buf[:, :n], accumulate=True)
    want = plain + bias.double() + old[:, :n].double()
    tol = (plain.abs() + bias.double().abs() + old[:, :n].double().abs()) * 2.0 ** -22
    if out_dtype == 1:
        tol = tol + want.abs() * 2.0 ** -8
    assert bool(((buf[:, :n].double() - want).abs() <= tol).all()) and torch.equal(buf[:, n:], old[:, n:])
