"""Rows of logits with a NaN or +inf next to masked entries: every number of the row is NaN, the
masked entries' own log probabilities too."""
import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab,top", [(4, 12, 12), (4, 100, 100), (1100, 40, 40), (4, 9001, 20), (2, 50257, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_entries_of_a_bad_row(rows, vocab, top, bad):
    say("logprobs bad rows", rows, vocab, top, bad)
    g = gq()
    z = torch.full((rows, vocab), float("-inf"))
    z[:, ::7] = torch.arange(len(z[0, ::7])) * 0.25
    z[0] = float("-inf")
    z[0, 3], z[0, 5] = bad, 1.0
    z[1, vocab - 1] = bad
    tokens = np.full(rows, 2, np.int64)
    tokens[1] = vocab - 1
    lp, h, ids, lps = (t.cpu().numpy() for t in g.token_logprobs(z.cuda(), torch.from_numpy(tokens).cuda(), top))
    rlp, rh, rids, rlps = lm.logprobs(z.numpy(), tokens, top)
    assert np.isnan(lps[:2]).all() and np.isnan(lp[:2]).all() and np.isnan(h[:2]).all()
    assert np.array_equal(ids, rids)
    eps = (vocab / 256 + 64) * 2.0 ** -22
    with np.errstate(invalid="ignore"):
        same = lambda a, b, e: (a == b) | (np.isnan(a) & np.isnan(b)) | (np.abs(a - b) <= e)  # noqa: E731
        assert same(lps, rlps, eps + np.abs(rlps) * 2.0 ** -22).all()
        assert same(lp, rlp, eps + np.abs(rlp) * 2.0 ** -22).all()
        assert same(h, rh, eps * (1 + np.abs(rh))).all()
