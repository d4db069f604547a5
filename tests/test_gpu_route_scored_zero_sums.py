"""Sigmoid scores that float64's 1 / (1 + exp(-l)) has as 0 (logits below -709.78): renormalised weights of such picks
alone are 0, and so is their gradient."""
import numpy as np
import pytest
import torch

from test_gpu_route_scored import DEV, U, gradient, run, scores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("depth", [700.0, 709.0, 710.0, 720.0, 740.0, 746.0, 2000.0])
def test_no_weights_no_gradient(depth):
    import routing_grouped_expert_gemm_amd as mok
    T, E, k = 8, 64, 4
    rng = np.random.default_rng(int(depth))
    l = (rng.random((T, E)) * 0.25 - depth).astype(np.float32)
    l[-1, 3] = 1.0                                         # a row with one score
    idx, w = run(l, k, None, "sigmoid")
    p = np.take_along_axis(scores(l, "sigmoid"), idx, 1)
    zero = p.sum(1) == 0
    # the logits lie within 0.25 above -depth: all of a row's below -709.79, all above -709.77, or either
    assert not zero[-1] and (depth <= 710.04 or zero[:-1].all()) and (depth >= 709.77 or not zero.any())
    assert (w[zero] == 0).all() and (w[~zero] > 0).any(1).all()
    dw = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.empty(T, E, device=DEV)
    mok.mok_topk_scored_backward(torch.from_numpy(l).to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(dw).to(DEV), out)
    torch.cuda.synchronize()
    o = out.cpu().numpy()
    assert (o[zero] == 0).all()
    with np.errstate(over="ignore"):
        ref, mag = gradient(l[~zero], idx[~zero], dw[~zero], "sigmoid", True, 1.0)
    assert (np.abs(o[~zero] - ref) <= 8 * U * mag + 1e-40).all()
