"""Tokens that name an expert more than once ("an expert named twice counts twice"), which gives an expert more
rows than there are tokens: in the integer form (at most 4 tokens, or at most 2 routes an expert on average), the
bf16 form and the form of one token's routes, all experts and a share, K of one body and of several. Bounds of
test_gpu_w4.py."""
import numpy as np
import pytest
import torch

from test_gpu_w4 import DEV, dev, half_step, layer_weights, moe, routing

pytestmark = pytest.mark.gpu

CASES = [  # T, d, I, E, e0, E_l, k, group
    (1, 512, 128, 8, 0, 8, 2, 32), (1, 512, 128, 8, 0, 8, 2, 128), (1, 2048, 1408, 64, 0, 64, 6, 128),
    (1, 2048, 1408, 64, 8, 20, 6, 128), (1, 256, 4224, 12, 2, 6, 5, 64), (2, 512, 256, 16, 0, 16, 2, 64),
    (3, 1152, 640, 48, 0, 48, 8, 128), (2, 7168, 256, 64, 0, 64, 8, 64), (3, 384, 1056, 7, 1, 5, 7, 32),
    (5, 256, 128, 8, 0, 8, 8, 32), (5, 256, 128, 100, 0, 100, 8, 32), (8, 640, 384, 6, 0, 6, 3, 128),
    (8, 2048, 4224, 4, 1, 2, 4, 64), (15, 512, 1152, 8, 0, 8, 5, 64), (15, 128, 2112, 90, 40, 30, 9, 32),
    (15, 7168, 128, 3, 0, 3, 3, 128)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,d,I,E,e0,E_l,k,group", CASES)
def test_repeated_picks(T, d, I, E, e0, E_l, k, group, zeros):
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(T * 17 + d + k)
    L = layer_weights(g, E_l, d, I, group, zeros)
    layer = mok.MoeW4Layer(*(dev(L[n]) for n in ("gate", "up", "down")), E=E, k=k, e0=e0, max_tokens=T)
    x, y_in = torch.randn(T, d, generator=g).bfloat16(), torch.randn(T, d, generator=g).bfloat16()
    rng = np.random.default_rng(T + k)
    idx, tw = routing(rng, T, E, k)
    half = idx.copy()
    half[:, :(k + 1) // 2] = e0 + E_l - 1
    for rows in (np.full_like(idx, e0), half, np.repeat(idx[:, :1], k, 1), e0 + rng.integers(0, 2, idx.shape).astype(np.int32) % E_l):
        layer.workspace.fill_(0xFF)                          # NaN wherever something unwritten is read
        ref, tol = moe(x, rows, tw, L, e0, group, y_in)
        buf = torch.full((T * d + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
        y = buf[:T * d].view(T, d)
        ix, w = torch.from_numpy(rows).to(DEV), torch.from_numpy(tw).to(DEV)
        layer.forward(x.to(DEV), ix, w, y, y_in=y_in.to(DEV))
        y2 = torch.empty_like(y)
        layer.forward(x.to(DEV), ix, w, y2, y_in=y_in.to(DEV))
        torch.cuda.synchronize()
        off = np.abs(y.double().cpu().numpy() - ref) - (tol + half_step(torch.bfloat16) * np.abs(ref))
        assert (off <= 0).all(), off.max()
        assert (buf[T * d:] == 7).all() and torch.equal(y, y2)
