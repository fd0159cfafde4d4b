"""The most rows of a call on logits: one less than a launch of 256 threads a row cannot hold."""
import pytest
import torch

from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu

MOST = (1 << 24) - 1


def test_more_rows_are_refused():
    say("too many rows")
    g = gq()
    lib, ctx = g._lib, g.context()
    buf = torch.zeros(64, device="cuda")
    p, n = buf.data_ptr(), MOST + 1
    assert lib.gq_token_logprobs(ctx.handle, p, 0, n, 3, 3, p, 1.0, 0, p, p, None, None, None) == g.EINVAL
    assert lib.gq_distill_loss(ctx.handle, p, 0, n, 3, 3, p, p, 1, 1.0, 0, None, p, None, None, 0, None) == g.EINVAL
    assert lib.gq_distill_grad(ctx.handle, p, 0, n, 3, 3, p, p, 1, 1.0, 0, p, None, p, 3, None) == g.EINVAL
    assert "rows" in lib.gq_last_error(ctx.handle).decode()


def test_most_rows():
    """Rows of three entries: the last 1023 have the bits that they have in a call of their own.  They
    begin on a line of 128 bytes, so that each lies in its lines as in the whole: which entries a
    thread adds goes by that."""
    say("most rows of logits")
    g = gq()
    rows = MOST
    z = torch.empty(rows, 3, device="cuda", dtype=torch.bfloat16).normal_(generator=torch.Generator("cuda").manual_seed(1))
    tokens = torch.arange(rows, device="cuda") % 3
    got = g.token_logprobs(z, tokens, 2)
    last = slice(rows - 1023, rows)
    some = z[last].clone()
    want = g.token_logprobs(some, tokens[last].clone(), 2)
    assert all(torch.equal(a[last], b) for a, b in zip(got, want))
    ids, lps = got[2][:, :1].contiguous(), got[3][:, :1].contiguous()
    loss, stats = g.distill_loss(z, ids, lps, tail=True)
    grad = g.distill_grad(z, ids, lps, 1.0, True, stats)
    want = g.distill_loss(some, ids[last].clone(), lps[last].clone(), tail=True, row_weight=torch.ones(1023, device="cuda"))
    assert torch.equal(loss[last], want[0]) and torch.equal(grad[last], want[1])
