"""Microscaled 4-bit matrices on the GPU against the 64-bit definitions: codes and scales bit for
bit, products within the rounding of their fp32 sums, refusals."""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_helpers import dev, gq, host, say

pytestmark = pytest.mark.gpu


def _make(rows, cols, dtype, seed):
    """Values over many scales, a zero block, exact grid points and ties among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-20, 20, (rows, -(-cols // 32))).repeat(32, 1)[:, :cols]
    pick = rng.random((rows, cols))
    x = np.where(pick < 0.1, rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, -0.0], (rows, cols)), x)
    x[rng.random((rows, cols)) < 0.05] = 0
    if cols >= 64:
        x[rows // 2, 32:64] = 0
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return t


def _check(x, rounding, seed=0, worker=0, index_base=0, t=None):
    g = gq()
    xd = t if t is not None else x.cuda()
    q, qt = g.mx_quantize(xd, rounding, seed=seed, worker=worker, index_base=index_base, by_cols=True)
    v = x.float().numpy().astype(np.float64)
    r = lm.draws(*v.shape, seed, worker, index_base) if rounding else None
    for packed, val, d in ((q, v, r), (qt, v.T, None if r is None else r.T)):
        codes, scales = lm.quantize(val, rounding, d)
        assert np.array_equal(host(packed.scales), scales)
        assert np.array_equal(host(packed.codes), codes)
        with np.errstate(over="ignore"):      # 4 * 2^126 is above both types' range: infinite
            want = lm.decode(codes, scales, val.shape[1]).astype(np.float32).astype(np.float64)
        for out in (g.BF16, g.F32):
            got = g.mx_dequantize(packed, out).double().cpu().numpy()
            assert np.array_equal(got, want, equal_nan=True)
    return q, qt


SHAPES = [(1, 1), (1, 31), (3, 33), (5, 257), (32, 64), (64, 256), (129, 515), (33, 1031)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rounding", [0, 1])
def test_quantize(rows, cols, dtype, rounding):
    say("mx quantize", rows, cols, dtype, rounding)
    _check(_make(rows, cols, dtype, rows * 1000 + cols), rounding, seed=2 ** 40 + cols, worker=3, index_base=12345)


@pytest.mark.parametrize("rounding", [0, 1])
def test_quantize_strided_rows(rounding):
    """Rows of a wider buffer that start at odd elements, and what lies between them untouched."""
    say("mx strided", rounding)
    g = gq()
    wide = _make(40, 301, torch.bfloat16, 7)
    x = wide[:, :270]
    xd = wide.cuda()[:, :270]
    _check(x.contiguous(), rounding, seed=5, t=xd)
    q, _ = g.mx_quantize(xd)
    out = torch.full((40, 301), 7.0, dtype=torch.bfloat16, device="cuda")
    g.mx_dequantize(q, out=out[:, :270])
    assert torch.equal(out[:, :270], g.mx_dequantize(q)) and bool((out[:, 270:] == 7).all())


def test_every_bf16_value():
    """Each finite bf16 value rounded under each scale that a larger companion sets."""
    say("mx every bf16")
    bits = np.arange(0, 0x7F80, dtype=np.uint16)
    vals = np.concatenate([bits, bits | 0x8000])
    x = torch.from_numpy(vals.view(np.int16).copy()).view(torch.bfloat16).view(-1, 32)
    _check(x, 0)
    up = torch.from_numpy((np.minimum(bits.astype(np.int64) + 0x180, 0x7F7F)).astype(np.int16)).view(torch.bfloat16)
    pair = torch.zeros(bits.size // 8, 32, dtype=torch.bfloat16)
    pair[:, 0::4] = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).view(-1, 8)
    pair[:, 1] = up.view(-1, 8).float().amax(1).to(torch.bfloat16)
    for rounding in (0, 1):
        _check(pair, rounding, seed=9)


def test_subnormal_and_extreme_blocks():
    say("mx extremes")
    x = torch.zeros(6, 64)
    x[0, :4] = torch.tensor([1e-45, -1e-40, 3e-39, 1.1e-38])
    x[1, :3] = torch.tensor([3.4028234663852886e38, -1e38, 2e37])
    x[2, 5] = float("inf")
    x[3, 40] = float("nan")
    x[4, :3] = torch.tensor([2.0 ** -125, 2.0 ** -127, 1.5 * 2.0 ** -126])
    x[5, 33:36] = torch.tensor([2.0 ** -126, 1.75 * 2.0 ** -126, -(2.0 ** -149)])
    for rounding in (0, 1):
        _check(x, rounding, seed=1)


def _bound(a, b, k):
    """Worst rounding of fp32 sums of k products taken 64 at a time: |a| |b| times the steps."""
    return (np.abs(a) @ np.abs(b).T) * (k / 64 + 64) * 2.0 ** -24


def _operands(m, n, k, seed):
    rng = np.random.default_rng(seed)
    a = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32))
    b = torch.from_numpy((rng.standard_normal((n, k)) * 0.1).astype(np.float32))
    return a, b


PRODUCTS = [(1, 1, 1), (1, 130, 100), (3, 17, 257), (16, 513, 1000), (9, 40, 9000), (2, 300, 5000), (17, 513, 1000), (33, 128, 32),
            (64, 200, 4100), (65, 31, 513), (128, 128, 256), (257, 300, 768), (300, 1031, 520),
            (700, 2100, 300), (2048, 2304, 512), (2100, 2050, 777),
            (4000, 3900, 777), (40, 300, 9000), (100, 90, 40000)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(m, n, k):
    say("mx matmul", m, n, k)
    g = gq()
    a, b = _operands(m, n, k, m + n + k)
    qa, qb = g.mx_quantize(a.cuda())[0], g.mx_quantize(b.cuda())[0]
    va = g.mx_dequantize(qa, g.F32).cpu().numpy().astype(np.float64)
    vb = g.mx_dequantize(qb, g.F32).cpu().numpy().astype(np.float64)
    ref = va @ vb.T
    bound = _bound(va, vb, k)
    got = g.mx_matmul(qa, qb, out_dtype=g.F32).cpu().numpy()
    assert np.all(np.abs(got - ref) <= bound)
    got16 = g.mx_matmul(qa, qb).float().cpu().numpy()
    assert np.all(np.abs(got16 - ref) <= bound + np.abs(ref) * 2.0 ** -8)
    # rows that the call packs: the same numbers
    assert torch.equal(g.mx_matmul(a.cuda(), qb, out_dtype=g.F32).cpu(), torch.from_numpy(got))
    a16 = a.to(torch.bfloat16).cuda()
    assert torch.equal(g.mx_matmul(a16, qb), g.mx_matmul(g.mx_quantize(a16)[0], qb))


@pytest.mark.parametrize("m,n,k", [(1, 40, 96), (20, 70, 600), (130, 300, 256)])
@pytest.mark.parametrize("out_dtype", [0, 1])
def test_matmul_bias_accumulate_and_strides(m, n, k, out_dtype):
    say("mx epilogue", m, n, k, out_dtype)
    g = gq()
    a, b = _operands(m, n, k, 5)
    qb = g.mx_quantize(b.cuda())[0]
    wide = torch.randn(m, k + 5).cuda()
    wide[:, :k] = a.cuda()
    bias = torch.randn(n).cuda()
    plain = g.mx_matmul(a.cuda(), qb, out_dtype=g.F32).double()
    old = torch.randn(m, n + 3).to(torch.float32 if out_dtype == 0 else torch.bfloat16).cuda()
    out = old.clone()
    g.mx_matmul(wide[:, :k], qb, bias=bias, out_dtype=out_dtype, out=out[:, :n], accumulate=True)
    want = plain + bias.double() + old[:, :n].double()
    # two more fp32 additions, and the type's own rounding
    tol = (plain.abs() + bias.double().abs() + old[:, :n].double().abs()) * 2.0 ** -22
    if out_dtype == 1:
        tol = tol + want.abs() * 2.0 ** -8
    assert bool(((out[:, :n].double() - want).abs() <= tol).all())
    assert torch.equal(out[:, n:], old[:, n:])


@pytest.mark.parametrize("m", [2, 40, 200])
def test_matmul_bad_blocks_and_extreme_scales(m):
    say("mx nan", m)
    g = gq()
    a, b = _operands(m, 150, 300, 6)
    a[1, 40] = float("inf")
    b[3, 290] = float("nan")
    a[0] *= 2.0 ** 100
    b[5] *= 2.0 ** -110
    b[6] = 0
    out = g.mx_matmul(g.mx_quantize(a.cuda())[0], g.mx_quantize(b.cuda())[0], out_dtype=g.F32).cpu().numpy()
    bad = np.zeros(out.shape, bool)
    bad[1], bad[:, 3] = True, True
    assert np.array_equal(np.isnan(out), bad)
    va = lm.decode(*lm.quantize(a.numpy()[:1], 0), 300)
    vb = lm.decode(*lm.quantize(b.numpy()[[0, 5, 6]], 0), 300)
    assert np.all(np.abs(out[0, [0, 5, 6]] - (va @ vb.T)[0]) <= _bound(va, vb, 300)[0])


def test_training_products_match_the_formulas():
    """dX = dY W and dW = dY^T X from operands by rows and by columns."""
    say("mx backward")
    g = gq()
    rng = np.random.default_rng(8)
    dy, w, x = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
                for s in ((77, 130), (130, 201), (77, 201)))
    q, qt = g.mx_quantize(dy, 1, seed=3, by_cols=True)
    wt, xt = g.mx_quantize(w, by_rows=False, by_cols=True)[1], g.mx_quantize(x, by_rows=False, by_cols=True)[1]
    for got, a, b in ((g.mx_matmul(q, wt, out_dtype=g.F32), q, wt), (g.mx_matmul(qt, xt, out_dtype=g.F32), qt, xt)):
        va, vb = (g.mx_dequantize(t, g.F32).cpu().numpy().astype(np.float64) for t in (a, b))
        assert np.all(np.abs(got.cpu().numpy() - va @ vb.T) <= _bound(va, vb, a.cols))


def test_empty_and_one_row():
    say("mx empty")
    g = gq()
    q, qt = g.mx_quantize(torch.empty(0, 40, device="cuda"), by_cols=False)
    assert q.rows == 0 and qt is None
    b = g.mx_quantize(torch.ones(7, 40, device="cuda"))[0]
    assert tuple(g.mx_matmul(q, b).shape) == (0, 7)
    assert tuple(g.mx_matmul(torch.empty(0, 40, device="cuda"), b).shape) == (0, 7)


def test_side_stream_and_graph():
    """A call on another stream than the default, captured and replayed with new inputs."""
    say("mx graph")
    g = gq()
    ctx = g.Context()
    b = g.mx_quantize(torch.randn(300, 512).cuda())[0]
    x = torch.randn(40, 512, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(40, 300, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.mx_matmul(x, b, out=out, ctx=ctx)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        g.mx_matmul(x, b, out=out, ctx=ctx)
    for i in range(3):
        x.copy_(torch.randn(40, 512))
        want = g.mx_matmul(x, b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_refusals():
    say("mx refusals")
    g = gq()
    x = torch.zeros(4, 64, device="cuda")
    b = g.mx_quantize(x)[0]
    lib, ctx = g._lib, g.context()

    def code(st):
        return st, lib.gq_last_error(ctx.handle).decode()

    def quant(**kw):
        a = dict(x=x.data_ptr(), dt=0, rows=4, cols=64, ld=64, rd=0, base=0, c=b.codes.data_ptr(),
                 s=b.scales.data_ptr(), ct=None, st=None)
        a.update(kw)
        return lib.gq_mx_quantize(ctx.handle, a["x"], a["dt"], a["rows"], a["cols"], a["ld"], a["rd"], 0, 0,
                                  a["base"], a["c"], a["s"], a["ct"], a["st"], None)

    assert quant(dt=2) == g.EINVAL and quant(rd=2) == g.EINVAL and quant(ld=63) == g.EINVAL
    assert quant(rows=-1) == g.EINVAL and quant(cols=0) == g.EINVAL and quant(cols=(1 << 23) + 1, ld=1 << 24) == g.EINVAL
    assert quant(s=None) == g.EINVAL and quant(c=None, s=None) == g.EINVAL and quant(x=None) == g.EINVAL
    assert quant(x=x.data_ptr() + 4) == g.EALIGN and quant(c=b.codes.data_ptr() + 8) == g.EALIGN
    assert quant(rd=1, base=2 ** 32 - 255) == g.EINVAL
    with pytest.raises(ValueError):
        g.mx_matmul(x[:, :32], b)
    with pytest.raises(ValueError):
        g.mx_quantize(x.T)
    with pytest.raises(TypeError):
        g.mx_quantize(x.double())
    with pytest.raises(ValueError):
        g.MXTensor(b.codes, b.scales, 257)
    o = torch.empty(4, 4, device="cuda")

    def mul(**kw):
        a = dict(a=x.data_ptr(), dt=0, sa=None, lda=64, M=4, N=4, K=64, bias=None, acc=0, od=0, o=o.data_ptr(), ldo=4)
        a.update(kw)
        return lib.gq_mx_matmul(ctx.handle, a["a"], a["dt"], a["sa"], a["lda"], b.codes.data_ptr(),
                                b.scales.data_ptr(), a["M"], a["N"], a["K"], a["bias"], a["acc"], a["od"], a["o"],
                                a["ldo"], None)

    assert mul(dt=3) == g.EINVAL and mul(dt=2) == g.EINVAL and mul(sa=b.scales.data_ptr()) == g.EINVAL
    assert mul(lda=63) == g.EINVAL and mul(ldo=3) == g.EINVAL and mul(K=0) == g.EINVAL and mul(N=0) == g.EINVAL
    assert mul(acc=2) == g.EINVAL and mul(od=2) == g.EINVAL and mul(o=o.data_ptr() + 4) == g.EALIGN
    st, msg = code(mul(o=None))
    assert st == g.EINVAL and "out" in msg
    assert lib.gq_mx_pitch(0) == 0 and lib.gq_mx_pitch(1) == 8 and lib.gq_mx_pitch(257) == 16
