"""Sizes that lead to every form of the tiled kernels around a model's layers, and the library's own
rules, compiled for the host, that say which."""
import ctypes
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "allreduce_compatible_gradient_amd", "csrc")

# (batch, shorter side, longer side) of updates: (tile of the Gram matrix, whether its sums are split,
# tile of its square, tile of the update); "128+" is the tile that has a CU of its own
UPDATES = {
    (1, 65, 66): ("64", False, "64", "64"),
    (1, 67, 1501): ("64", True, "64", "64"),
    (30, 65, 513): ("64", False, "64", "128"),
    (12, 201, 4101): ("64", True, "64", "256"),
    (48, 385, 769): ("128", False, "64", "64"),
    (64, 201, 1501): ("128+", False, "64", "128"),
    (43, 65, 8003): ("128+", True, "64", "128"),
    (64, 257, 769): ("192", False, "64", "64"),
    (43, 129, 4101): ("192", True, "64", "64"),
    (64, 385, 769): ("256", False, "64", "128"),
    (43, 201, 8003): ("256", True, "64", "128"),
    (30, 600, 601): ("128", False, "128", "128"),
    (16, 600, 603): ("128+", False, "128+", "128"),
    (24, 513, 515): ("192", False, "192", "64"),
    (30, 700, 769): ("256", False, "256", "128"),
    (12, 768, 2304): None,
    (24, 768, 768): None,
    (1, 2048, 2048): None,
    (1, 4100, 4301): None,
}

# (M, N, K) of 8-bit products of more than 16 rows: (side of the tile, whether K is split)
PRODUCTS = {
    (17, 31, 200): (64, False),
    (70, 1003, 300): (64, False),
    (33, 257, 8000): (64, True),
    (65, 129, 4100): (64, True),
    (129, 11008, 65): (128, False),
    (131, 11009, 200): (128, False),
    (385, 5003, 384): (128, False),
    (1025, 8001, 65): (256, False),
    (1027, 8003, 200): (256, False),
    (2049, 4096, 513): (256, False),
}

SHIM = """
#include "gq_plans.h"
extern "C" void update_form(int64_t batch, int64_t n, int64_t m, int *f) {
  const gq::Side g = gq::gram_plan(batch, n, m), s = gq::symmetric_plan(batch, n, gq::up64(n) / 64, false);
  f[0] = g.side; f[1] = g.alone; f[2] = g.splits; f[3] = s.side; f[4] = s.alone; f[5] = gq::update_side(batch, n, m);
  f[6] = gq::ortho_is_small(n, m);
}
extern "C" void product_form(int64_t M, int64_t N, int64_t K, int *f) {
  const gq::I8Plan p = gq::i8_plan(M, N, K);
  f[0] = p.bm; f[1] = p.bn; f[2] = p.splits;
}
"""


def rules(folder):
    """(form of an update, form of a product) by the library's header."""
    with open(os.path.join(folder, "forms.cpp"), "w") as f:
        f.write(SHIM)
    lib = os.path.join(folder, "forms.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, os.path.join(folder, "forms.cpp"), "-o", lib], check=True)
    dll = ctypes.CDLL(lib)

    def call(f, *sizes):
        out = (ctypes.c_int * 8)()
        f(*[ctypes.c_int64(s) for s in sizes], out)
        return list(out)

    def update(batch, n, m):
        g, alone, splits, s, s_alone, u, small = call(dll.update_form, batch, n, m)[:7]
        assert not small
        name = lambda side, by_itself: "128+" if side == 128 and by_itself else str(side)  # noqa: E731
        return name(g, alone), splits > 1, name(s, s_alone), str(u)

    def product(m, n, k):
        bm, bn, splits = call(dll.product_form, m, n, k)[:3]
        assert (bm, bn) in ((64, 128), (128, 128), (256, 256))
        return bm, splits > 1

    return update, product
