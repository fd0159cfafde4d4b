"""Language-model operators at the edges of their launches: rows as long as a block's slice holds,
and as many rows as a packed matrix may have."""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_helpers import gq, host, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [131008, 131009, 131072])
def test_longest_slices(vocab):
    """1025 rows: as few slices a row as there may be, beginning at every place of a line.  A thread
    adds vocab / 256 terms, and some 64 roundings follow: (vocab / 256 + 64) 2^-22 covers the
    logarithm's error as an absolute one."""
    say("longest slices", vocab)
    g = gq()
    rows, ld = 1025, 131077
    buf = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(vocab))
    z = buf[:, :vocab]
    tokens = torch.arange(rows, device="cuda") * 127 % vocab
    lp, h, ids, lps = g.token_logprobs(z, tokens, 9)
    some = list(range(0, 8)) + [63, 64, 1024]
    rlp, rh, rids, rlps = lm.logprobs(z[some].float().cpu().numpy(), tokens[some].cpu().numpy(), 9, 1.0)
    eps = (vocab / 256 + 64) * 2.0 ** -22
    assert np.all(np.abs(lp[some].cpu().numpy() - rlp) <= eps + np.abs(rlp) * 2.0 ** -22)
    assert np.all(np.abs(h[some].cpu().numpy() - rh) <= eps * (1 + np.abs(rh)))
    assert np.array_equal(ids[some].cpu().numpy(), rids)
    assert np.all(np.abs(lps[some].cpu().numpy() - rlps) <= eps + np.abs(rlps) * 2.0 ** -22)


@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 65473), (torch.float32, 70001), (torch.bfloat16, 131009)])
@pytest.mark.parametrize("tail", [False, True])
def test_long_rows_of_one_slice(dtype, vocab, tail):
    """Rows that registers do not hold and that are so many that none is cut: a context of its own,
    whose scratch memory no other call has brought to size."""
    say("long rows", dtype, vocab, tail)
    g = gq()
    rows, top = 1030, 5
    gen = torch.Generator("cuda").manual_seed(vocab)
    z = torch.empty(rows, vocab, dtype=dtype, device="cuda").normal_(generator=gen)
    ids = torch.arange(rows * top, device="cuda", dtype=torch.int32).reshape(rows, top) * 13 % vocab
    lps = torch.log_softmax(torch.empty(rows, top + 1, device="cuda").normal_(generator=gen), 1)[:, :top].contiguous()
    ctx = g.Context()
    w = torch.ones(rows, device="cuda")
    loss, grad = g.distill_loss(z, ids, lps, 1.0, tail, row_weight=w, ctx=ctx)
    some = [0, 1, 511, 1029]
    rl, rg, _ = lm.distill(z[some].float().cpu().numpy(), ids[some].cpu().numpy(), lps[some].cpu().numpy(), 1.0, tail)
    eps = (vocab / 256 + 64) * 2.0 ** -22
    assert np.all(np.abs(loss[some].cpu().numpy() - rl) <= eps + np.abs(rl) * 2.0 ** -22)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    assert np.all(np.abs(grad[some].double().cpu().numpy() - rg) <= (2 * eps + half) * np.abs(rg).max())
    again, stats = g.distill_loss(z, ids, lps, 1.0, tail, ctx=g.Context())
    assert torch.equal(again, loss)
    assert torch.equal(g.distill_grad(z, ids, lps, 1.0, tail, stats, w), grad)


def test_most_rows():
    """2^23 rows of one element, both ways: the codes by columns are those of the transpose by rows."""
    say("most rows")
    g = gq()
    n = 1 << 23
    x = torch.randn(n, 1, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    q, qt = g.mx_quantize(x, by_cols=True)
    flat, _ = g.mx_quantize(x.reshape(1, n))
    assert torch.equal(qt.codes, flat.codes) and torch.equal(qt.scales, flat.scales)
    last = slice(n - 300, n)
    codes, scales = lm.quantize(x[last].cpu().numpy().astype(np.float64), 0, None)
    assert np.array_equal(host(q.codes)[last], codes) and np.array_equal(host(q.scales)[last], scales)
