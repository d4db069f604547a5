"""Weights of the choice by scores are float64 values, rounded once, whatever the rule and whether or not a row is
near a border: 2^-24 of the weight, and 2^-33 for both sides' float64 (a row's exponentials are held to 2^-35)."""
import numpy as np
import pytest

from test_gpu_route_scored import U, choose, logits, run

pytestmark = pytest.mark.gpu


def close(l, k, bias, score, G, Gk, top, renorm, scale):
    idx, w = run(l, k, bias, score, G, Gk, top, renorm, scale)
    ri, rw = choose(l, bias, k, score, G, Gk, top, renorm, scale)
    assert np.array_equal(idx, ri)
    assert (np.abs(w - rw) <= U * (1 + 2.0 ** -9) * np.abs(rw) + 2.0 ** -149).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k,G,Gk", [(16, 3, 1, 1), (64, 6, 1, 1), (100, 8, 4, 2), (256, 8, 8, 4), (384, 7, 1, 1), (512, 8, 16, 5), (520, 9, 4, 2)])
def test_one_rounding(E, k, G, Gk, renorm, score):
    rng = np.random.default_rng(E)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for spread in (0.1, 1.0, 6.0, 40.0):
        l = (spread * logits(rng, 60, E)).astype(np.float32)
        # rows near a border: equal logits, some of them one float32 apart
        l[:20, 1::2] = l[:20, 0:E - 1:2]
        l[10:20, 1::4] = np.nextafter(l[10:20, 1::4], np.float32(np.inf))
        for b in (None, bias):
            close(l, k, b, score, G, Gk, 2, renorm, 1.0)
