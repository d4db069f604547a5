"""Picks that a bias has taken from far below the row's largest logit, where their softmax is nothing in float64:
renormalised over the picks it is still exp(l) / sum exp(l), in every form of the choice, and its gradient goes with
it. Weights: one rounding, 2^-24, and 2^-40 for float64's exponentials; gradients as in test_gpu_route_scored.py."""
import numpy as np
import pytest
import torch

from test_gpu_route_scored import DEV, U, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k,G,Gk", [(64, 6, 1, 1), (256, 8, 8, 4), (600, 5, 1, 1), (640, 6, 4, 2), (64, 12, 1, 1)])
def test_softmax_of_far_picks(E, k, G, Gk):
    import routing_grouped_expert_gemm_amd as mok
    rng = np.random.default_rng(E + k)
    T = 30
    for depth in (100.0, 700.0, 720.0, 740.0, 1000.0, 5000.0):
        l = rng.standard_normal((T, E)).astype(np.float32)
        ids = np.sort(rng.permutation(E // G * Gk)[:k])
        bias = np.zeros(E, np.float32)
        bias[ids] = 4 + np.arange(k, 0, -1)                            # picked, in this order
        l[:, ids] -= np.float32(depth)
        l[::3, ids[0]] = l[::3, ids[1]]
        if k > 2:
            bias[ids[2]] = bias[ids[1]]                                # a tie of scores that are 0
        idx, w = run(l, k, bias, "softmax", G, Gk, 1, True, 1.0)
        assert (np.sort(idx, 1) == ids).all()
        p = np.take_along_axis(l, idx, 1).astype(np.float64)
        p = np.exp(p - p.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        assert (np.abs(w - p) <= U * (1 + 2.0 ** -16) * p).all(), depth
        dw = rng.standard_normal((T, k)).astype(np.float32)
        out = torch.empty(T, E, device=DEV)
        mok.mok_topk_scored_backward(torch.from_numpy(l).to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(dw).to(DEV),
                                     out, score="softmax", renorm=True)
        torch.cuda.synchronize()
        dot = (p * dw).sum(1, keepdims=True)
        ref, mag = np.zeros((T, E)), np.zeros((T, E))
        np.put_along_axis(ref, idx.astype(np.int64), p * (dw - dot), 1)
        np.put_along_axis(mag, idx.astype(np.int64), p * (np.abs(dw) + (p * np.abs(dw)).sum(1, keepdims=True)), 1)
        assert (np.abs(out.cpu().numpy() - ref) <= 8 * U * mag).all(), depth
