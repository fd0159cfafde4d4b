"""The resource report covers the kernels around a model's layers (CPU only; another file's checks of
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
    for k in ("k_i8_rows", "k_i8_tops", "k_i8_both", "k_i8_matmul", "k_i8_matmul_few", "k_i8_join", "k_embed",
              "k_embed_sort", "k_embed_rows", "k_embed_join", "k_ortho_norm", "k_ortho_start", "k_ortho_symmetric",
              "k_ortho_join", "k_ortho_update", "k_ortho_small"):
        assert k in names, k


def test_tiles_keep_two_waves(resources):
    """A tile's loop covers one wave's waits with another's products: two waves a SIMD at least, but for
    the form whose blocks have a CU each, which goes by four buffers instead."""
    for k, v in resources.items():
        if "Li2ELi2ELi4ELi4ELi4E" in k:
            continue
        if "k_i8_matmul" in k or "k_ortho_symmetric" in k or "k_ortho_update" in k:
            assert v["Occupancy"] >= 2, k
