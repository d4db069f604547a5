"""Groups whose two best members have biases of opposite signs, so that float32 worths have lost what tells the groups
apart: the picks are those of float64 (test_gpu_route_scored.py), whose own worths are off by 2^-53 of the biases, far
less than what lies between any two of these."""
import numpy as np
import pytest

from test_gpu_route_scored import check, choose, logits, scores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,Gk", [(16, 8, 3), (64, 8, 4), (60, 5, 2), (256, 8, 4), (240, 16, 7), (512, 16, 5), (20, 10, 4)])
def test_worths_that_cancel(E, G, Gk, score):
    n = E // G
    for size, spread in ((1000.0, 1e-3), (1000.0, 1.0), (30.0, 1e-5), (8.0, 1e-6), (1e6, 1.0)):
        rng = np.random.default_rng(E + int(size))
        l = (spread * logits(rng, 200, E)).astype(np.float32)
        bias = np.full(E, -size, np.float32)
        bias[::n] = size
        c = np.sort((scores(l, score) + bias).reshape(200, G, n), axis=2)[:, :, -2:].sum(2)
        far = np.diff(np.sort(c, axis=1), axis=1).min(1) > 2.0 ** -50 * size
        if score == "softmax" and size > 1e3:
            far &= False                                   # (float64 holds too little of such a score)
        if far.any():
            check(l[far], min(4, Gk * n), bias, score, G, Gk)
            bias[1::n] = np.float32(-size) * np.float32(1 + 2.0 ** -20)      # and biases that do not quite cancel
            c = np.sort((scores(l, score) + bias).reshape(200, G, n), axis=2)[:, :, -2:].sum(2)
            far &= np.diff(np.sort(c, axis=1), axis=1).min(1) > 2.0 ** -50 * size
            check(l[far], min(4, Gk * n), bias, score, G, Gk)


@pytest.mark.parametrize("E,G,Gk", [(64, 8, 3), (60, 5, 2), (256, 8, 4)])
def test_worths_past_float32(E, G, Gk):
    """Biases whose sum only float64 holds: the groups of largest sum have the highest ids, or the lowest sums do."""
    rng = np.random.default_rng(E)
    n = E // G
    for sign in (1, -1):
        bias = np.repeat(sign * np.linspace(1.8e38, 3.2e38, G), n).astype(np.float32)
        bias += (1e36 * rng.random(E)).astype(np.float32)
        check(logits(rng, 40, E), 4, bias, "sigmoid", G, Gk)
        check(logits(rng, 40, E), 4, bias, "softmax", G, Gk, renorm=False)
