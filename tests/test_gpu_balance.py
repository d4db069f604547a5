"""The router's balance loss (mok_balance_loss, mok_balance_loss_backward) against its definition
in float64.

Tolerances. A probability is exp(l - m) / sum: the exponent's argument is rounded (relative error
of the exponential |l - m| 2^-24 for the subtraction and as much for the factor log2 e), and the
exponential, the sum and the quotient add a few units each, so p is off by at most
u = (16 + 2 |l - m|) 2^-24 of itself; the sums over tokens add up to the longest chain of 40
additions. mean_prob and the loss inherit that (all terms are positive). A gradient element
c p (f - sum f p) is a difference: it is off by at most 4 u of c p (f + sum f p)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def reference(logits, idx, off, k, alpha, dloss=1.0):
    """loss, counts, mean_prob, dlogits and the gradient's scale c p (f + sum f p), in float64."""
    lg = logits.double().numpy()
    T, E = lg.shape
    off = [0, T] if off is None else [min(max(int(v), 0), T) for v in off]
    S = len(off) - 1
    loss, counts, mean = 0.0, np.zeros((S, E), np.int32), np.zeros((S, E))
    dl, scale = np.zeros((T, E)), np.zeros((T, E))
    for s in range(S):
        a, b = off[s], off[s + 1]
        if b <= a:
            continue
        x = lg[a:b]
        m = x.max(1, keepdims=True)
        p = np.exp(x - np.where(np.isfinite(m), m, 0.0))
        tot = p.sum(1, keepdims=True)
        p = np.divide(p, tot, out=np.zeros_like(p), where=tot > 0)
        i = idx[a:b].numpy()
        i = i[(i >= 0) & (i < E)]
        counts[s] = np.bincount(i, minlength=E)
        f = counts[s] * (E / (k * (b - a)))
        mean[s] = p.mean(0)
        loss += alpha / S * (f * mean[s]).sum()
        dot = (p * f).sum(1, keepdims=True)
        c = dloss * alpha / (S * (b - a))
        dl[a:b], scale[a:b] = c * p * (f - dot), abs(c) * p * (f + dot)
    return loss, counts, mean, dl, scale


def run(mok, logits, idx, off, k, alpha, dloss=1.0, bufs=None):
    T, E = logits.shape
    S = 1 if off is None else len(off) - 1
    lg, ix = logits.to(DEV), idx.to(DEV)
    so = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    ws = torch.full((mok.mok_balance_loss_workspace_bytes(T, E, S),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    loss, counts = torch.full((1,), 7.0, device=DEV), torch.full((S, E), -9, dtype=torch.int32,
                                                                 device=DEV)
    mean, dl = torch.full((S, E), 7.0, device=DEV), torch.full((T, E), 7.0, device=DEV)
    mok.mok_balance_loss(lg, ix, alpha, loss, counts, mean, ws, seq_offsets=so)
    mok.mok_balance_loss_backward(lg, counts, k, alpha, torch.tensor([dloss], device=DEV), dl,
                                  seq_offsets=so)
    torch.cuda.synchronize()
    return [t.cpu() for t in (loss, counts, mean, dl)]


def check(got, ref, spread):
    u = (16 + 2 * spread + 40) * 2.0 ** -24
    loss, counts, mean, dl = got
    rl, rc, rm, rd, scale = ref
    assert np.array_equal(counts.numpy(), rc)
    assert abs(float(loss) - rl) <= 2 * u * abs(rl)
    assert (np.abs(mean.numpy() - rm) <= u * rm + 1e-37).all()
    assert (np.abs(dl.numpy() - rd) <= 4 * u * scale + 1e-37).all()


CASES = [  # T, E, k, offsets
    (1, 1, 1, None), (1, 8, 2, None), (7, 5, 5, None), (257, 8, 2, None), (1000, 64, 6, None),
    (333, 60, 4, None), (100, 63, 3, None), (75, 100, 6, None), (64, 128, 8, None),
    (50, 130, 8, None), (97, 256, 8, None), (40, 255, 8, None), (33, 384, 8, None),
    (20, 500, 8, None), (9, 1000, 16, None), (5, 1024, 64, None), (3, 1021, 64, None),
    (40000, 16, 2, None),
    (500, 64, 6, [0, 500]), (500, 64, 6, [0, 1, 1, 17, 17, 17, 400, 480]),   # padding behind
    (500, 64, 6, [3, 10, 499]), (100, 20, 4, [0, 0, 0, 100, 100]), (64, 8, 2, [5, 5, 5]),
    (5000, 32, 4, [0, 15, 16, 32, 33, 2000, 4999]), (37, 7, 3, list(range(38))),
    (300, 64, 6, [-5, 100, 900]),
]


@pytest.mark.parametrize("T,E,k,off", CASES)
def test_against_float64(T, E, k, off):
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = torch.randn(T, E, generator=g) + torch.randn(1, E, generator=g)
    idx = torch.topk(logits, k, dim=1).indices.int()
    ref = reference(logits, idx, off, k, 0.01, dloss=-3.0)
    got = run(mok, logits, idx, off, k, 0.01, dloss=-3.0)
    check(got, ref, 14.0)
    again = run(mok, logits, idx, off, k, 0.01, dloss=-3.0)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,E,off", [(512, 8, None), (300, 5, [0, 7, 7, 200, 290]), (33, 1, None),
                                     (5000, 64, None)])
def test_equal_counts_leave_no_gradient(T, E, off):
    """k = E: every count is the mean one and the gradient zero, exactly. With one pick less it is
    off by at most 4 u of c p (|g| + sum |g| p), g = f - E (mean count) / (k n): g is one rounding off
    and nothing cancels but it."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn(T, E, generator=g) * 2
    idx = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).int()
    assert not run(mok, logits, idx, off, E, 0.01)[3].any()
    idx[3, 0] = -1
    dl = run(mok, logits, idx, off, E, 0.01)[3].numpy()
    _, counts, _, rd, _ = reference(logits, idx, off, E, 0.01)
    bounds = [0, T] if off is None else off
    p = torch.softmax(logits.double(), 1).numpy()
    spread = float((logits.amax(1) - logits.amin(1)).max())
    u = (16 + 2 * spread + 40) * 2.0 ** -24
    for s, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a < b:
            gs = np.abs(counts[s] / (b - a) - 1.0)
            scale = 0.01 / ((len(bounds) - 1) * (b - a)) * p[a:b] * (gs + (p[a:b] * gs).sum(1, keepdims=True))
            assert (np.abs(dl[a:b] - rd[a:b]) <= 4 * u * scale + 1e-15 * 0.01 / (b - a)).all()


def test_masked_logits_and_invalid_picks():
    """-inf logits, the type's lowest value, a row of nothing but -inf, picks outside [0, E) and a
    pick named twice; tokens of no sequence may hold anything, NaN included."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(5)
    for E in (12, 13):
        T, k = 90, 3
        logits = torch.randn(T, E, generator=g)
        logits[::3, 4:] = -float("inf")
        logits[1::7, :2] = torch.finfo(torch.float32).min
        logits[10] = -float("inf")
        logits[11] = torch.finfo(torch.float32).min
        idx = torch.randint(0, E, (T, k), generator=g).int()
        idx[3, 0], idx[4, 1], idx[5] = -1, E, torch.tensor([2, 2, 2])
        off = [2, 40, 80]
        logits[:2], logits[80:] = float("nan"), float("inf")
        idx[81] = 2 ** 31 - 1
        inside = logits.clone()
        inside[:2] = inside[80:] = 0.0
        got = run(mok, logits, idx, off, k, 0.5)
        check(got, reference(inside, idx, off, k, 0.5), 14.0)
        assert torch.equal(got[3][:2], torch.zeros(2, E)) and not got[3][80:].any()
        assert not got[3][10].any()


def test_nan_and_infinity_reach_their_row():
    import routing_grouped_expert_gemm_amd as mok
    for bad in (float("nan"), float("inf")):
        logits = torch.zeros(20, 8)
        logits[7, 3] = bad
        idx = torch.zeros(20, 1, dtype=torch.int32)
        loss, counts, mean, dl = run(mok, logits, idx, None, 1, 1.0)
        assert torch.isnan(loss).all() and torch.isnan(mean).all() and int(counts.sum()) == 20
        assert torch.isnan(dl[7]).all() and torch.isfinite(dl[:7]).all()


def test_gradient_against_differences():
    """Central differences of the library's own loss; the loss's picks are held fixed. With step
    h the difference quotient is off by the third derivative (h^2 / 6 of terms at most alpha E)
    and by the loss's rounding over h: with h = 2^-5, alpha = 8, E = 6: 2^-10 / 6 * 48 * 1.5 is
    0.012 at the most, the rounding 2^-22 * loss / h below 1e-4."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(9)
    T, E, k, h = 3, 6, 2, 2.0 ** -5
    logits = torch.randn(T, E, generator=g)
    idx = torch.topk(logits, k, dim=1).indices.int()
    dl = run(mok, logits, idx, None, k, 8.0)[3]
    for t in range(T):
        for e in range(E):
            up, dn = logits.clone(), logits.clone()
            up[t, e] += h
            dn[t, e] -= h
            d = (run(mok, up, idx, None, k, 8.0)[0] - run(mok, dn, idx, None, k, 8.0)[0]) / (2 * h)
            assert abs(float(d) - float(dl[t, e])) <= 0.012


def test_no_tokens():
    import routing_grouped_expert_gemm_amd as mok
    loss, counts, mean, dl = run(mok, torch.zeros(0, 6), torch.zeros(0, 2, dtype=torch.int32),
                                 [0, 0, 0], 2, 1.0)
    assert float(loss) == 0.0 and not counts.any() and not mean.any() and dl.shape == (0, 6)


def test_counts_match_the_dispatch_plan():
    """The loss's counts are the plan's when all experts are local."""
    import routing_grouped_expert_gemm_amd as mok
    T, E, k = 512, 64, 6
    g = torch.Generator().manual_seed(2)
    logits = torch.randn(T, E, generator=g)
    idx = torch.topk(logits, k, dim=1).indices.int()
    counts = run(mok, logits, idx, None, k, 1.0)[1]
    i32 = dict(dtype=torch.int32, device=DEV)
    c, o = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    ws = torch.empty(mok.mok_dispatch_plan_workspace_bytes(T, k, E), dtype=torch.uint8, device=DEV)
    mok.mok_dispatch_plan(idx.to(DEV), E, 0, E, T, c, o, torch.empty((E, 1), **i32),
                          torch.empty(T * k, **i32), ws)
    torch.cuda.synchronize()
    assert torch.equal(counts[0], c.cpu())


def test_unaligned_rows():
    """logits and dlogits that do not start on 16 bytes (a view one element into a buffer)."""
    import routing_grouped_expert_gemm_amd as mok
    T, E, k = 65, 8, 2
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(T, E, generator=g)
    idx = torch.topk(logits, k, dim=1).indices.int()
    ref = run(mok, logits, idx, None, k, 0.1)
    buf = torch.zeros(T * E + 1, device=DEV)
    view = buf[1:].view(T, E)
    view.copy_(logits)
    out = torch.empty(T * E + 1, device=DEV)
    dl = out[1:].view(T, E)
    mok.mok_balance_loss_backward(view, ref[1].to(DEV), k, 0.1, torch.ones(1, device=DEV), dl)
    torch.cuda.synchronize()
    check([ref[0], ref[1], ref[2], dl.cpu()], reference(logits, idx, None, k, 0.1), 14.0)


def test_graph_replays():
    """Captured once and replayed on new inputs, with eager work between the replays."""
    import routing_grouped_expert_gemm_amd as mok
    T, E, k, off = 700, 64, 6, [0, 100, 650]
    g = torch.Generator().manual_seed(4)
    so = torch.tensor(off, dtype=torch.int32, device=DEV)
    lg, ix = torch.zeros(T, E, device=DEV), torch.zeros(T, k, dtype=torch.int32, device=DEV)
    ws = torch.empty(mok.mok_balance_loss_workspace_bytes(T, E, 2), dtype=torch.uint8, device=DEV)
    loss, mean = torch.empty(1, device=DEV), torch.empty(2, E, device=DEV)
    counts, dl = torch.empty(2, E, dtype=torch.int32, device=DEV), torch.empty(T, E, device=DEV)
    one = torch.ones(1, device=DEV)

    def step():
        mok.mok_balance_loss(lg, ix, 0.01, loss, counts, mean, ws, seq_offsets=so)
        mok.mok_balance_loss_backward(lg, counts, k, 0.01, one, dl, seq_offsets=so)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        logits = torch.randn(T, E, generator=g)
        idx = torch.topk(logits, k, dim=1).indices.int()
        eager = run(mok, logits, idx, off, k, 0.01)
        lg.copy_(logits)
        ix.copy_(idx)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (loss, counts, mean, dl)):
            assert torch.equal(a, b.cpu())
