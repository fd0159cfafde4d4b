"""The resource report covers the language-model kernels (CPU only; the other file's checks of
spills hold for every kernel of the report)."""
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RES = os.path.join(ROOT, "allreduce_compatible_gradient_amd", "_build", "kernel_resources.json")


@pytest.fixture(scope="module")
def resources():
    if not os.path.exists(RES):
        pytest.skip("the library has not been built here (no resource report)")
    with open(RES) as f:
        return json.load(f)


def test_report_covers_the_kernels(resources):
    names = " ".join(resources)
    for k in ("k_mx_rows", "k_mx_both", "k_mx_dequantize", "k_mx_matmul", "k_mx_join",
              "k_mx_matmul_few", "k_logprobs", "k_logprobs_join", "k_distill_row",
              "k_distill_slices", "k_distill_join", "k_distill_grad"):
        assert k in names, k


def test_held_rows_keep_three_blocks(resources):
    """A CU holds three blocks of 256 threads and 26 chunks, two of the 256 x 256 tiles' waves."""
    for k, v in resources.items():
        if "k_distill_row" in k and "Li26E" in k:
            assert v["Occupancy"] >= 3, k
        if "k_mx_matmul" in k and "few" not in k:
            assert v["Occupancy"] >= 2, k
