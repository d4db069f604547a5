"""What the 4-bit products keep of x and of the experts' hidden values: a value next to a far larger one of its
group, whose code is the zero point, and hidden values that cancel but for their last bits. All sums here are whole
numbers that float32 holds in any order, so that the results have to be equal."""
import numpy as np
import pytest
import torch

from test_gpu_w4 import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 4, 7])
def test_small_values_by_large_ones(M, group, zeros):
    import routing_grouped_expert_gemm_amd as mok
    N, K = 40, 640
    g = torch.Generator().manual_seed(M + group)
    x = torch.randint(-255, 256, (M, K), generator=g).float()          # 8 bits: bf16 holds them
    x[:, ::group] = 2.0 ** 28
    q = torch.randint(0, 16, (N, K), generator=g)
    z = torch.randint(0, 16, (N, K // group), generator=g) if zeros else torch.full((N, K // group), 8)
    q[:, ::group] = z                                                  # the large values' codes
    ref = x.double() @ (q - z.repeat_interleave(group, 1)).double().T
    if M > 4:                                                          # x q - z x: 2^28 (15 - 15) rounds
        x[:, ::group] = 0
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8)
    out = torch.empty(M, N, device=DEV)
    mok.mok_w4_gemm(x.bfloat16().to(DEV), codes.to(DEV), torch.ones(N, K // group, device=DEV).bfloat16(), out,
                    zeros=z.to(torch.uint8).to(DEV) if zeros else None)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().double(), ref)


def pack(v):
    """Values -8 .. 7 as codes of zero point 8."""
    q = (v + 8).to(torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4)


HIDDEN = [(1, 4, 2, 128), (1, 64, 4, 64), (3, 8, 2, 32), (4, 2, 1, 128)]          # T, E, k, group: integers


ROWS = [(5, 2, 1, 128), (8, 1, 1, 64), (20, 4, 2, 32), (70, 8, 2, 128), (600, 4, 2, 64)]      # bf16


@pytest.mark.parametrize("T,E,k,group", HIDDEN + ROWS)
def test_hidden_values_that_cancel(T, E, k, group):
    """H = [2^18 + 2^9 + 2, 2^18 + 2^9, 2^25 (code: the zero point)] 2^j, for token j; weights 1, -1, 0: y is 2^(j + 1)."""
    import routing_grouped_expert_gemm_amd as mok
    d, I = 2 * group, 2 * group
    up, gate, down = (torch.zeros(E, *s, dtype=torch.int64) for s in ((I, d), (I, d), (d, I)))
    for c in range(0, I, group):                           # in each group of H
        up[:, c, 0], up[:, c, 1], up[:, c + 1, 0], up[:, c + 5, 0] = 1, 1, 1, 1
        up[:, c:c + 2, 4] = 1
        gate[:, c:c + 2, 2], gate[:, c + 5, 3] = 1, 1
    down[:, :, 0], down[:, :, 1] = 1, -1
    if T > 4:
        gate[:, 5::group] = 0                              # the integers' case alone
    x = torch.zeros(T, d)
    for t in range(T):
        x[t, :5] = torch.tensor([2.0 ** 11, 2.0 ** -6, 2.0 ** 7, 2.0 ** 14, 4.0])
        x[t, [0, 1, 4]] *= 2.0 ** (t % 8)
    one = lambda a: torch.ones(*a.shape[:-1], a.shape[-1] // group, device=DEV).bfloat16()  # noqa: E731
    L = [(pack(a).to(DEV), one(a), None) for a in (gate, up, down)]
    layer = mok.MoeW4Layer(*L, E=E, k=k, max_tokens=T)
    idx = torch.stack([(torch.arange(k) + t) % E for t in range(T)]).to(torch.int32).to(DEV)
    tw = torch.full((T, k), 1.0 / k, device=DEV)
    y = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    layer.forward(x.bfloat16().to(DEV), idx, tw, y)
    torch.cuda.synchronize()
    ref = torch.tensor([2.0 ** (1 + t % 8) for t in range(T)]).double()[:, None].expand(T, d)
    assert torch.equal(y.cpu().double(), ref)
