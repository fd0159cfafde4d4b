"""The example's draws: no two of its stochastic roundings share a key."""
import importlib.util
import os

import pytest

from tests.gpu_helpers import gq, say

pytestmark = pytest.mark.gpu


def test_no_key_serves_twice(monkeypatch):
    say("example keys")
    g = gq()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_mx.py")
    spec = importlib.util.spec_from_file_location("distill_mx", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    keys = []
    quantize, fused = g.mx_quantize, g.fused_mean

    def mx_quantize(x, rounding=g.MX_NEAREST, seed=0, worker=0, *a, **kw):
        if rounding == g.MX_STOCHASTIC:
            keys.append((seed, worker))
        return quantize(x, rounding, seed, worker, *a, **kw)

    def fused_mean(flat, *a, seed, **kw):
        keys.extend((seed, k) for k in range(len(flat)))    # worker k draws with (seed, k)
        return fused(flat, *a, seed=seed, **kw)

    monkeypatch.setattr(g, "mx_quantize", mx_quantize)
    monkeypatch.setattr(g, "fused_mean", fused_mean)
    ex.run(steps=4, workers=3, tokens=64, width=64, hidden=64, vocab=257, top=8, say=None)
    assert len(keys) == 4 * (3 * 2 + 3)
    assert len(set(keys)) == len(keys), sorted(k for k in keys if keys.count(k) > 1)
