"""8-bit matrices with a scale for each row, through the library, against the 64-bit definitions:
codes and scales equal, products within their fp32 roundings."""
import numpy as np
import pytest
import torch

from oracle import layers, lm
from tests.gpu_helpers import dev, gq, host, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def values(rows, cols, seed, dtype=F32):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 12, (rows, 1)))
    x[:, rng.random(cols) < 0.05] *= 16
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def check_codes(q, x, rounding, r, rows, cols):
    codes, scales = layers.quantize(x, rounding, r)
    assert q.rows == rows and q.cols == cols
    assert np.array_equal(host(q.scales), scales, equal_nan=True)
    assert np.array_equal(host(q.codes), codes)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 128), (5, 129), (4, 2048), (2, 2049), (3, 12288), (2, 12289),
                                       (130, 257), (64, 512), (65, 513), (1, 40000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("stochastic", [False, True])
def test_quantise_by_rows(rows, cols, dtype, stochastic):
    say("int8 rows", rows, cols, dtype, stochastic)
    g = gq()
    x = values(rows, cols, rows * 31 + cols, dtype)
    r = lm.draws(rows, cols, 77, 3, 5) if stochastic else None
    q, none = g.int_quantize(x.cuda(), g.INT_STOCHASTIC if stochastic else g.INT_NEAREST, 77, 3, 5)
    assert none is None
    check_codes(q, x.float().numpy(), int(stochastic), r, rows, cols)


@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 1), (1, 300), (128, 128), (129, 127), (200, 515), (63, 1024), (517, 130)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("by_rows", [False, True])
def test_quantise_by_columns_and_both_ways(rows, cols, dtype, stochastic, by_rows):
    say("int8 columns", rows, cols, dtype, stochastic, by_rows)
    g = gq()
    x = values(rows, cols, rows * 17 + cols, dtype)
    x[:, cols // 2] = 0
    r = lm.draws(rows, cols, 9, 0, 0) if stochastic else None
    q, qt = g.int_quantize(x.cuda(), int(stochastic), 9, by_rows=by_rows, by_cols=True)
    check_codes(qt, x.float().numpy().T, int(stochastic), None if r is None else r.T, cols, rows)
    if by_rows:
        check_codes(q, x.float().numpy(), int(stochastic), r, rows, cols)
    else:
        assert q is None


def test_borders():
    """Ties to even, the largest code, values next to ties, tiny and huge rows, what is not finite."""
    say("int8 borders")
    g = gq()
    x = np.zeros((12, 133), np.float32)
    x[0, :8] = [127, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5]
    x[1, :6] = [127, np.nextafter(np.float32(0.5), np.float32(1)), np.nextafter(np.float32(0.5), np.float32(0)),
                np.nextafter(np.float32(-63.5), np.float32(0)), 63.5, -0.0]
    x[2, 3] = 1e-37      # inv is not finite
    x[3, 132] = 4e-37    # inv is
    x[3, 0] = -1.5e-37
    x[4] = 3.4e38
    x[5, 7] = np.nan
    x[6, 132], x[6, 0] = -np.inf, 3
    x[7] = -1e-45
    x[8, 100] = 5
    x[9, :3] = [1, -1 / 254, 1 / 254]
    x[10] = np.linspace(-3, 3, 133)
    q, qt = g.int_quantize(torch.from_numpy(x).cuda(), by_cols=True)
    check_codes(q, x, 0, None, 12, 133)
    check_codes(qt, x.T, 0, None, 133, 12)
    r = lm.draws(12, 133, 5)
    q, qt = g.int_quantize(torch.from_numpy(x).cuda(), g.INT_STOCHASTIC, seed=5, by_cols=True)
    check_codes(q, x, 1, r, 12, 133)
    check_codes(qt, x.T, 1, r.T, 133, 12)
    alone, _ = g.int_quantize(torch.from_numpy(x).cuda())
    check_codes(alone, x, 0, None, 12, 133)


def test_rows_of_a_wider_matrix():
    """Row strides, rows that begin at any element, and outputs given by the caller, whose neighbours
    stay as they were."""
    say("int8 strides")
    g = gq()
    wide = values(70, 400, 3, BF16).cuda()
    for width in (257, 399):
        x = wide[:, :width]
        q, qt = g.int_quantize(x, by_cols=True)
        check_codes(q, x.float().cpu().numpy(), 0, None, 70, width)
        check_codes(qt, x.float().cpu().numpy().T, 0, None, width, 70)
    big = torch.full((9, 128), 55, dtype=torch.int8, device="cuda")
    scales = torch.full((12,), -1.0, device="cuda")
    out = g.IntTensor(big[:5], scales[:5], 100)
    g.int_quantize(values(5, 100, 4).cuda(), out=out)
    assert torch.all(big[5:] == 55) and torch.all(scales[5:] == -1)


# ----------------------------------------------------------------------------- products
def product_case(m, n, k, seed):
    rng = np.random.default_rng(seed)
    a, sa = layers.quantize(rng.standard_normal((m, k)).astype(np.float32), 0)
    b, sb = layers.quantize((rng.standard_normal((n, k)) * 0.02).astype(np.float32), 0)
    return a, sa, b, sb, rng.standard_normal(n).astype(np.float32)


def check_product(got, a, sa, b, sb, bias, old=None):
    """float(sum) sa sb: three roundings; the bias and the old value one more each of what they make;
    a bf16 half a step more.  Each rounding is off by at most 2^-24 of its result."""
    want, mag = layers.matmul(a, sa, b, sb, bias)
    bound = (3 * mag + (0 if bias is None else np.abs(want))) * 2.0 ** -24
    if old is not None:
        want = want + old
        bound = bound + np.abs(want) * 2.0 ** -24
    if got.dtype == BF16:
        bound = bound * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8
    d = np.abs(got.double().cpu().numpy() - want)
    assert np.all(d <= bound * (1 + 1e-6) + 1e-44), (d - bound).max()


def packed(g, codes, scales, cols):
    return g.IntTensor(dev(codes), dev(scales), cols)


SIZES = [(1, 1, 1), (1, 17, 127), (2, 48, 128), (16, 33, 129), (16, 100, 4000), (17, 31, 65), (40, 130, 640), (64, 128, 256),
         (65, 129, 257), (100, 700, 100), (257, 300, 384), (300, 2000, 2100), (33, 257, 8000), (1000, 1029, 200)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("form", ["plain", "bias", "accumulate", "both"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product(m, n, k, form, dtype):
    say("int8 product", m, n, k, form, dtype)
    g = gq()
    a, sa, b, sb, bias = product_case(m, n, k, m + n + k)
    bias = bias if form in ("bias", "both") else None
    out, old = None, None
    if form in ("accumulate", "both"):
        out = torch.randn(m, n, generator=torch.Generator().manual_seed(m)).to(dtype).cuda()
        old = out.double().cpu().numpy()
    got = g.int_matmul(packed(g, a, sa, k), packed(g, b, sb, k), bias=None if bias is None else dev(bias),
                       out_dtype=g.BF16 if dtype == BF16 else g.F32, out=out, accumulate=out is not None)
    check_product(got, a, sa, b, sb, bias, old)


@pytest.mark.parametrize("m,n,k", [(2048, 4224, 384), (2304, 4096, 257), (700, 9000, 128)])
def test_largest_tiles(m, n, k):
    say("int8 largest tiles", m, n, k)
    g = gq()
    a, sa, b, sb, bias = product_case(m, n, k, 5)
    for dtype, code in ((F32, g.F32), (BF16, g.BF16)):
        check_product(g.int_matmul(packed(g, a, sa, k), packed(g, b, sb, k), out_dtype=code), a, sa, b, sb, None)
        check_product(g.int_matmul(packed(g, a, sa, k), packed(g, b, sb, k), bias=dev(bias), out_dtype=code), a, sa, b, sb, bias)


@pytest.mark.parametrize("m,n,k", [(1, 50, 4096), (1, 20, 131072), (3, 40, 300), (7, 70, 4000), (16, 40, 2048), (16, 33, 2049),
                                   (16, 20, 12289), (33, 65, 513), (130, 140, 1100)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_quantises_its_rows(m, n, k, dtype):
    """Rows in fp32 or bf16 give the bits of the packed rows."""
    say("int8 product of rows", m, n, k, dtype)
    g = gq()
    _, _, b, sb, bias = product_case(1, n, k, 8)
    x = values(m, k, 9, dtype).cuda()
    q, _ = g.int_quantize(x)
    w = packed(g, b, sb, k)
    for out in (g.F32, g.BF16):
        assert torch.equal(g.int_matmul(x, w, out_dtype=out, bias=dev(bias)), g.int_matmul(q, w, out_dtype=out, bias=dev(bias)))
    check_product(g.int_matmul(x, w, out_dtype=g.F32), host(q.codes)[:, :q.codes.shape[1]], host(q.scales), b, sb, None)


def test_longest_sums():
    """131072 products of 127 * 127 stay within 32 bits, with one sign and with both."""
    say("int8 longest sums")
    g = gq()
    k = 1 << 17
    for m in (1, 17, 40):
        a, b = np.full((m, k), 127, np.int8), np.full((5, k), 127, np.int8)
        b[1] = -127
        b[2, ::2] = -127
        sa, sb = np.ones(m, np.float32), np.array([1, 1, 1, 0, np.nan], np.float32)
        got = g.int_matmul(packed(g, a, sa, k), packed(g, b, sb, k), out_dtype=g.F32).cpu().numpy()
        assert np.all(got[:, :4] == np.array([k * 16129, -k * 16129, 0, 0], np.float32)) and np.all(np.isnan(got[:, 4]))


@pytest.mark.parametrize("m", [1, 16, 50])
def test_rows_without_numbers(m):
    """A row of A that is NaN makes its row NaN alone; a zero row gives the bias."""
    say("int8 rows without numbers", m)
    g = gq()
    x = values(m, 200, 1)
    x[0, 5] = np.nan
    if m > 2:
        x[2] = 0
        x[m - 1, 199] = -np.inf
    _, _, b, sb, bias = product_case(1, 70, 200, 2)
    got = g.int_matmul(x.cuda(), packed(g, b, sb, 200), bias=dev(bias), out_dtype=g.F32)
    bad = torch.isnan(got).all(1).cpu()
    assert torch.equal(torch.isnan(got).any(1).cpu(), bad)
    assert bad.tolist() == [i == 0 or (m > 2 and i == m - 1) for i in range(m)]
    if m > 2:
        assert torch.equal(got[2].cpu(), torch.from_numpy(bias))


@pytest.mark.parametrize("m,n", [(5, 37), (40, 37), (300, 301)])
def test_rows_behind_the_last_stay(m, n):
    """Row strides of the output; what lies between and behind its rows is not written."""
    say("int8 output strides", m, n)
    g = gq()
    a, sa, b, sb, _ = product_case(m, n, 150, 6)
    for dtype in (F32, BF16):
        buf = torch.full((m + 3, n + 11), 7.0, dtype=dtype, device="cuda")
        got = g.int_matmul(packed(g, a, sa, 150), packed(g, b, sb, 150), out=buf[:m, :n], out_dtype=g.BF16 if dtype == BF16 else g.F32)
        check_product(got, a, sa, b, sb, None)
        assert torch.all(buf[m:] == 7) and torch.all(buf[:, n:] == 7)


def test_refusals():
    say("int8 refusals")
    g = gq()
    x = torch.zeros(4, 8, device="cuda")
    w = g.int_quantize(torch.ones(3, 8, device="cuda"))[0]
    none = g.int_quantize(torch.zeros(0, 8, device="cuda"))[0]
    assert none.rows == 0 and g.int_matmul(none, w).shape == (0, 3) and g.int_matmul(x[:0], w).shape == (0, 3)
    for call in (lambda: g.int_matmul(torch.zeros(4, 9, device="cuda"), w),
                 lambda: g.int_matmul(x, w, accumulate=True),
                 lambda: g.int_matmul(x, w, bias=torch.zeros(2, device="cuda")),
                 lambda: g.int_matmul(x, w, out=torch.zeros(4, 4, device="cuda"), out_dtype=g.F32),
                 lambda: g.int_quantize(torch.zeros(8, 4, device="cuda").T),
                 lambda: g.int_quantize(x, out=w),
                 lambda: g.IntTensor(w.codes, w.scales, 200),
                 lambda: g.IntTensor(w.codes, w.scales[:2], 8)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.int_quantize(x.half()), lambda: g.int_quantize(x.cpu()),
                 lambda: g.int_matmul(x, w, out=torch.zeros(4, 3, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: g.int_quantize(x, rounding=2),
                 lambda: g.int_quantize(x, by_rows=False),
                 lambda: g.int_quantize(x, g.INT_STOCHASTIC, index_base=2 ** 32 - 31),
                 lambda: g.int_quantize(torch.zeros(1, (1 << 17) + 1, device="cuda")),
                 lambda: g.int_quantize(torch.zeros((1 << 17) + 1, 1, device="cuda"), by_rows=False, by_cols=True),
                 lambda: g.int_matmul(x, w, accumulate=2, out=torch.zeros(4, 3, device="cuda"), out_dtype=5),
                 lambda: g.int_quantize(torch.zeros(40, device="cuda")[1:33].view(4, 8))):
        with pytest.raises((g.GQError, ValueError, TypeError)):
            call()
