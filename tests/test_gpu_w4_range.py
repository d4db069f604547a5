"""4-bit products whose scales and values of x lie far apart, and results near float32's largest value: what fits is
there, with the bound of test_gpu_w4.py. A group's sum of x and its codes is formed before its scale and has to
fit as well, which every case here does."""
import numpy as np
import pytest
import torch

from test_gpu_w4 import DEV, dev, half_step, layer_weights, moe, product, routing, weight

pytestmark = pytest.mark.gpu

CASES = [(-100, 104), (60, 58), (-128, 120), (100, -120), (-20, 100), (0, -126), (110, -80)]     # binades of x, of the scales


@pytest.mark.parametrize("M", [1, 3, 4, 5, 13, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_far_scales(M, group, zeros):
    import routing_grouped_expert_gemm_amd as mok
    N, K = 72, 256
    for bx, bs in CASES:
        g = torch.Generator().manual_seed(M + group + bx)
        x = (torch.randn(M, K, generator=g).clamp(-3, 3).double() * 2.0 ** bx).bfloat16()
        w = weight(g, (), N, K, group, zeros, 2.0 ** bs)
        ref, tol = product(x.double().numpy(), w, group)
        assert np.abs(ref).max() < 2.0 ** 128
        D = dev(w)
        out = torch.empty(M, N, device=DEV)
        mok.mok_w4_gemm(x.to(DEV), D[0], D[1], out, zeros=D[2])
        torch.cuda.synchronize()
        off = np.abs(out.double().cpu().numpy() - ref) - (tol + half_step(torch.float32) * np.abs(ref) + 2.0 ** -149)
        assert (off <= 0).all(), (bx, bs, off.max())


@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (3, 8, 2), (9, 4, 3)])
def test_far_scales_of_experts(T, E, k):
    """Down weights of 2^100 behind up weights of 2^-104."""
    import routing_grouped_expert_gemm_amd as mok
    d, I, group = 256, 128, 64
    g = torch.Generator().manual_seed(T)
    L = layer_weights(g, E, d, I, group, True)
    L["up"] = (L["up"][0], (L["up"][1].double() * 2.0 ** -104).bfloat16(), L["up"][2])
    L["down"] = (L["down"][0], (L["down"][1].double() * 2.0 ** 100).bfloat16(), L["down"][2])
    layer = mok.MoeW4Layer(*(dev(L[n]) for n in ("gate", "up", "down")), E=E, k=k, max_tokens=T)
    x = torch.randn(T, d, generator=g).bfloat16()
    idx, tw = routing(np.random.default_rng(T), T, E, k)
    y = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    layer.forward(x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(tw).to(DEV), y)
    torch.cuda.synchronize()
    ref, tol = moe(x, idx, tw, L, 0, group, None)
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol + half_step(torch.bfloat16) * np.abs(ref)).all()
