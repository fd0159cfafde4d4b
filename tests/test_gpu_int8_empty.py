"""8-bit matrices without rows: their columns have a scale each all the same."""
import pytest
import torch

from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1, 8, 300, 100001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rounding", [0, 1])
@pytest.mark.parametrize("by_rows", [False, True])
def test_columns_of_no_rows(cols, dtype, rounding, by_rows):
    """No element: a largest magnitude of zero, hence scales of zero, whatever the buffer held; its
    neighbours stay."""
    say("int8 of no rows", cols, dtype, rounding, by_rows)
    g = gq()
    scales = torch.full((cols + 40,), float("nan"), device="cuda")
    out = g.IntTensor.empty(cols, 0, "cuda")
    out.scales = scales[:cols]
    q, qt = g.int_quantize(torch.zeros(0, cols, dtype=dtype, device="cuda"), rounding, by_rows=by_rows, by_cols=True, out_t=out)
    assert qt is out and qt.rows == cols and qt.cols == 0 and qt.codes.shape == (cols, 0)
    assert torch.equal(qt.scales, torch.zeros(cols, device="cuda")) and torch.isnan(scales[cols:]).all()
    assert q is None or (q.rows == 0 and q.cols == cols)
    fresh = g.int_quantize(torch.zeros(0, cols, dtype=dtype, device="cuda"), rounding, by_rows=False, by_cols=True)[1]
    assert not fresh.scales.any()
