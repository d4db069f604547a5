"""Balance loss's gradient where nearly all experts have the same count.

A sequence of n equal tokens picks E - 1 of E experts, u is left out: f is E / (E - 1) for the picked ones
and 0 for u, and the gradient alpha / n p (f - sum f p) is alpha / n (E / (E - 1)) p p_u for the picked
ones, far below f p where p_u is small. The kernel counts f from the mean count to the nearest, f'. With
r = 2^-24: p comes from an exponential of an argument up to 10 (off by at most (10 / ln 2 + 2) r), a sum of
at most 64 and a quotient, 87 r of itself in all, and sum f' p from a tree of at most 12 roundings more: f'
- sum f' p is off by 100 r (|f'| + sum |f'| p), and the products by 200 r of themselves. One token: f' is
0 but for u, and that is 100 r p_u: every value keeps its relative accuracy."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("E", [3, 4, 6, 12, 20, 64])
def test_gradient_keeps_its_bits(E, n):
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(E)
    u, k = E // 2, E - 1
    row = 2 * torch.rand(E, generator=g) - 1
    row[u] = -8.5                                    # the unpicked expert is unlikely
    logits = row.repeat(n, 1).to(DEV)
    picks = torch.tensor([e for e in range(E) if e != u], dtype=torch.int32, device=DEV).repeat(n, 1)
    loss, counts = torch.empty(1, device=DEV), torch.empty(1, E, dtype=torch.int32, device=DEV)
    mean, dl = torch.empty(1, E, device=DEV), torch.empty(n, E, device=DEV)
    ws = torch.empty(mok.mok_balance_loss_workspace_bytes(n, E), dtype=torch.uint8, device=DEV)
    mok.mok_balance_loss(logits, picks, 1.0, loss, counts, mean, ws)
    mok.mok_balance_loss_backward(logits, counts, k, 1.0, torch.ones(1, device=DEV), dl)
    torch.cuda.synchronize()
    p = torch.softmax(row.double(), 0)
    f = torch.full((E,), E / (E - 1), dtype=torch.float64)
    f[u] = 0.0
    ref = p * p[u] * f / n
    ref[u] = -(E / (E - 1)) * p[u] * (1 - p[u]) / n
    c = torch.full((E,), float(n))
    c[u] = 0
    fm = (c - (n * k + E // 2) // E).abs().double() * E / (k * n)
    assert n > 1 or fm.sum() == fm[u]                # one token: nothing but u
    tol = 100 * (fm + (fm * p).sum()) * p / n + 200 * ref.abs()
    assert ((dl.cpu().double() - ref).abs() <= 2.0 ** -24 * tol).all()
