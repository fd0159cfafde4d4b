"""The sizes that the GPU tests run lead to every form that the library's rules choose (CPU only)."""
import pytest

from tests import layer_forms


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    return layer_forms.rules(str(tmp_path_factory.mktemp("forms")))


def test_updates(rules):
    for sizes, form in layer_forms.UPDATES.items():
        assert form is None or rules[0](*sizes) == form, (sizes, rules[0](*sizes))
    reached = [rules[0](*sizes) for sizes in layer_forms.UPDATES]
    assert {(f[0], f[1]) for f in reached} >= {("64", False), ("64", True), ("128", False), ("128+", False), ("128+", True),
                                               ("192", False), ("192", True), ("256", False), ("256", True)}
    assert {f[2] for f in reached} == {"64", "128", "128+", "192", "256"}
    assert {f[3] for f in reached} == {"64", "128", "256"}


def test_products(rules):
    for sizes, form in layer_forms.PRODUCTS.items():
        assert rules[1](*sizes) == form, (sizes, rules[1](*sizes))


def test_no_other_forms(rules):
    """Over a grid of sizes: a split Gram matrix has a CU a block, and only the smallest tiles of a product
    are split, so no form is left out above."""
    update, product = rules
    listed = {f[:2] for f in layer_forms.UPDATES.values() if f}
    for n in (65, 130, 257, 385, 520, 700, 1000, 1500, 2049, 3001, 4096):
        for m in (65, 300, 777, 1500, 2304, 4100, 8000, 20000, 65536):
            for batch in (1, 2, 5, 12, 24, 48, 200):
                if m >= n:
                    assert update(batch, n, m)[:2] in listed, (batch, n, m, update(batch, n, m))
    for m in (17, 64, 65, 200, 333, 1000, 2048, 5000, 8192, 100000):
        for n in (1, 100, 300, 1029, 4096, 11008, 50257, 131072):
            for k in (1, 128, 768, 3071, 4096, 11008, 131072):
                tile, split = product(m, n, k)
                assert tile == 64 or not split, (m, n, k)
