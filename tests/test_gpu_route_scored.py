"""The choice of experts by scores (mok_topk_scored, mok_route_scored) and its gradient against their
definitions in float64 (numpy).

The picks have to be equal. Scores of both sides are float64 and off by a few units of 2^-53, so
picks could differ only where two choices (or worths of groups) that are not equal lie within 1e-15 of
each other: the random inputs have none, and the planted ties are exact on both sides (equal logits
with equal bias).

Weights: float64 rounded once to float32; a softmax that is not renormalised may take its sum of
exponentials from float32 values, each off by at most 2 units of 2^-24: 4 * 2^-24 of the weight.
Gradients: the share of a pick is a difference of float64 values, rounded once; of a softmax as it is,
p (g - sum g p) with float32 p off by 4 units and the difference taken in float32: 8 * 2^-24 of
p (|g| + sum |g| p). dlogits_in adds one rounding: 2^-24 of the result."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def scores(l, kind):
    l = l.astype(np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    top = l.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.exp(l - np.where(np.isneginf(top), 0, top))
        s = p.sum(1, keepdims=True)
    return np.where(s > 0, p / np.where(s > 0, s, 1), np.where(np.isnan(s), np.nan, 0.0))


def choose(l, bias, k, kind, G, Gk, top, renorm, scale):
    """Row by row, by sorting."""
    T, E = l.shape
    s = scores(l, kind)
    c = s if bias is None else s + bias.astype(np.float64)
    out = np.isneginf(l) | (False if bias is None else np.isneginf(bias))
    idx, w = np.empty((T, k), np.int64), np.empty((T, k))
    for t in range(T):
        order = lambda ids, v: sorted(ids, key=lambda e: (0 if np.isnan(v[e]) else 1, -v[e], e))  # noqa: E731
        keep = list(range(E))
        if Gk < G:
            n = E // G
            worth = np.empty(G)
            for g in range(G):
                ids = [e for e in range(g * n, (g + 1) * n) if not out[t, e]]
                ids = order(ids, np.where(np.isnan(c[t]), np.nan, c[t]))[:top]
                worth[g] = -np.inf if not ids else sum(c[t, e] for e in ids)
            kept = order(range(G), worth)[:Gk]
            keep = [e for g in sorted(kept) for e in range(g * n, (g + 1) * n)]
        v = np.where(out[t], -np.inf, c[t])
        idx[t] = order(keep, v)[:k]
        p = s[t, idx[t]]
        tot = p.sum()
        w[t] = scale * (p if not renorm else p / tot if tot != 0 else 0 * p)
    return idx, w


def run(l, k, bias=None, score="sigmoid", G=1, Gk=1, top=2, renorm=True, scale=1.0):
    import routing_grouped_expert_gemm_amd as mok
    T = l.shape[0]
    ld = torch.from_numpy(np.ascontiguousarray(l)).to(DEV)
    bd = None if bias is None else torch.from_numpy(bias).to(DEV)
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, k), 7.0, device=DEV)
    mok.mok_topk_scored(ld, k, idx[:T], w[:T], score=score, bias=bd, n_groups=G, topk_groups=Gk,
                        group_top=top, renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    assert (idx[T] == -7).all() and (w[T] == 7).all()
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy()


def check(l, k, bias=None, score="sigmoid", G=1, Gk=1, top=2, renorm=True, scale=1.0):
    idx, w = run(l, k, bias, score, G, Gk, top, renorm, scale)
    ri, rw = choose(l, bias, k, score, G, Gk, top, renorm, scale)
    assert np.array_equal(idx, ri), np.argwhere((idx != ri).any(1))[:5]
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    ok = ~np.isnan(rw)
    assert (np.abs(w[ok] - rw[ok]) <= 4 * U * np.abs(rw[ok]) + 1e-45).all()


def logits(rng, T, E):
    return (rng.standard_normal((T, E)) + 0.5 * rng.standard_normal((1, E))).astype(np.float32)


RULES = [(1, 1, 1, 1, 1, 2), (3, 2, 2, 1, 1, 1), (5, 7, 3, 7, 3, 2), (17, 8, 8, 1, 1, 2),
         (9, 20, 4, 5, 2, 2), (33, 64, 6, 1, 1, 1), (40, 64, 6, 8, 3, 2), (16, 96, 7, 3, 2, 1),
         (65, 256, 8, 8, 4, 2), (66, 256, 8, 16, 5, 1), (31, 160, 6, 8, 3, 2), (18, 100, 5, 4, 2, 2),
         (10, 111, 3, 3, 1, 2), (12, 240, 8, 2, 1, 2), (7, 384, 8, 1, 1, 1), (7, 384, 8, 8, 4, 2),
         (5, 512, 16, 4, 3, 2), (5, 513, 8, 1, 1, 1), (4, 1024, 64, 32, 8, 2), (4, 1000, 9, 1, 1, 1),
         (6, 48, 17, 1, 1, 1), (3, 64, 64, 1, 1, 1), (300, 256, 1, 1, 1, 1), (9, 32, 4, 32, 6, 2)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,G,Gk,top", RULES)
def test_against_float64(T, E, k, G, Gk, top, score):
    rng = np.random.default_rng(T * 1000 + E)
    l, bias = logits(rng, T, E), (0.1 * rng.standard_normal(E)).astype(np.float32)
    check(l, k, bias, score, G, Gk, top, True, 2.5)
    check(l, k, None, score, G, Gk, top, True, 1.0)
    check(l, k, bias, score, G, Gk, top, False, 1.0)
    check(l, k, None, score, G, Gk, top, False, -0.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,Gk", [(64, 1, 1), (256, 8, 4), (60, 5, 2), (384, 1, 1), (1024, 8, 2)])
def test_ties_go_to_the_lower_id(E, G, Gk, score):
    rng = np.random.default_rng(E)
    k = 6
    coarse = np.round(2 * rng.standard_normal((40, E))).astype(np.float32) / 2
    bias = np.round(4 * rng.standard_normal(E)).astype(np.float32) / 64
    check(np.zeros((5, E), np.float32), k, None, score, G, Gk)
    check(np.full((3, E), -3.25, np.float32), k, np.zeros(E, np.float32), score, G, Gk)
    check(coarse, k, None, score, G, Gk)
    check(coarse, k, bias, score, G, Gk)
    check(np.where(coarse == 0, np.float32(-0.0), coarse), k, bias, score, G, Gk, 1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_neighbouring_values(score):
    """Logits one float32 apart, in every order: the float32 of their scores cannot tell them."""
    rng = np.random.default_rng(5)
    for base, E in ((1.5, 64), (-2.0, 256), (0.01, 384), (6.0, 48)):
        u = (np.float32(base).view(np.int32) + rng.permuted(np.tile(np.arange(E, dtype=np.int32), (20, 1)), axis=1))
        l = u.astype(np.int32).view(np.float32)
        for G, Gk in ((1, 1), (4, 2)):
            check(l, 5, None, score, G, Gk, 1)
            check(l, 5, np.zeros(E, np.float32), score, G, Gk)
            check(l, 5, np.full(E, 0.25, np.float32), score, G, Gk, 2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,Gk,k", [(64, 1, 1, 6), (256, 8, 4, 8), (20, 5, 2, 5), (640, 1, 1, 7), (96, 3, 1, 30)])
def test_experts_left_out(E, G, Gk, k, score):
    """-inf logits and biases: rows with some, with all but few, with whole groups and with nothing."""
    rng = np.random.default_rng(E + 1)
    l = logits(rng, 40, E)
    l[rng.random(l.shape) < 0.3] = -np.inf
    l[5:10][rng.random((5, E)) < 0.97] = -np.inf
    l[10], l[11], l[12, 1:], l[13, :-1] = -np.inf, -np.inf, -np.inf, -np.inf
    n = E // G
    l[14:20, :n], l[15:20, -n:] = -np.inf, -np.inf
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for renorm in (True, False):
        check(l, k, None, score, G, Gk, 2, renorm)
        check(l, k, bias, score, G, Gk, 2, renorm)
    bias[rng.random(E) < 0.4] = -np.inf
    check(logits(rng, 10, E), k, bias, score, G, Gk, 1)
    check(l, k, bias - 5, score, G, Gk, 2)


def test_ends_of_the_range():
    rng = np.random.default_rng(8)
    l = logits(rng, 20, 64)
    for scale in (1e-30, 1e-8, 12.0):
        check(l * np.float32(scale), 6, None, "softmax", renorm=True)
        check(l * np.float32(min(scale, 8.0)), 6, None, "sigmoid", renorm=True)
        check(l * np.float32(scale), 6, l[0], "softmax", renorm=False)
    far = np.full((4, 64), -2000.0, np.float32)          # scores that are zero in float64 too
    far[:, 3], far[1:, 60] = 0, -1000
    check(far, 4, None, "softmax")
    check(far + 30, 4, None, "sigmoid")


def test_not_a_number_shows():
    rng = np.random.default_rng(9)
    for E, G, Gk in ((64, 1, 1), (256, 8, 4), (600, 1, 1)):
        l = logits(rng, 6, E)
        l[1, 7] = np.nan
        l[3, E - 1] = np.nan
        idx, w = run(l, 4, None, "sigmoid", G, Gk)
        ri, _ = choose(l[[0, 2, 4, 5]], None, 4, "sigmoid", G, Gk, 2, True, 1.0)
        assert np.array_equal(idx[[0, 2, 4, 5]], ri)
        assert idx[1, 0] == 7 and idx[3, 0] == E - 1 and np.isnan(w[[1, 3]]).all()
        assert np.isfinite(w[[0, 2, 4, 5]]).all()
        _, w = run(l, 4, None, "softmax", G, Gk)
        assert np.isnan(w[[1, 3]]).any(1).all() and np.isfinite(w[[0, 2, 4, 5]]).all()
        l[1, 7], l[3] = np.inf, np.inf                   # sigmoid: a score of 1
        check(l, 4, None, "sigmoid", G, Gk)


def test_offsets_past_32_bits():
    import routing_grouped_expert_gemm_amd as mok
    T, E, k = (1 << 31) // 256 + 300, 256, 2
    l = torch.empty(T, E, device=DEV)
    l.normal_()
    idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    mok.mok_topk_scored(l, k, idx, w)
    dw = torch.ones(T, k, device=DEV)
    dw[:, 1] = -1
    mok.mok_topk_scored_backward(l, idx, dw, l_out := torch.empty_like(l))
    torch.cuda.synchronize()
    tail = slice(T - 200, T)
    ln = l[tail].cpu().numpy()
    ri, rw = choose(ln, None, k, "sigmoid", 1, 1, 2, True, 1.0)
    assert np.array_equal(idx[tail].cpu().numpy(), ri)
    assert np.abs(w[tail].cpu().numpy() - rw).max() <= 4 * U
    ref, scale = gradient(ln, ri, np.tile([1.0, -1.0], (200, 1)), "sigmoid", True, 1.0)
    assert (np.abs(l_out[tail].cpu().numpy() - ref) <= 8 * U * scale).all()


@pytest.mark.parametrize("T,d,E,k,dtype", [(1, 64, 256, 8, "bf16"), (130, 256, 64, 6, "bf16"), (33, 100, 20, 3, "fp32")])
def test_route_from_rows(T, d, E, k, dtype):
    """The logits are mok_route's, bit for bit; the picks those of mok_topk_scored on them."""
    import routing_grouped_expert_gemm_amd as mok
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(T)
    x, wr = torch.randn(T, d, generator=g).to(t).to(DEV), (torch.randn(E, d, generator=g) * d ** -0.5).to(t).to(DEV)
    lg = [torch.empty(T, E, device=DEV) for _ in range(2)]
    idx = [torch.empty(T, k, dtype=torch.int32, device=DEV) for _ in range(2)]
    w = [torch.empty(T, k, device=DEV) for _ in range(2)]
    bias = torch.randn(E, generator=g).to(DEV) * 0.1
    mok.mok_route(x, wr, k, lg[0], idx[0], w[0])
    mok.mok_route_scored(x, wr, k, lg[1], idx[1], w[1], bias=bias, n_groups=4, topk_groups=2, scale=2.5)
    mok.mok_topk_scored(lg[0], k, idx[0], w[0], bias=bias, n_groups=4, topk_groups=2, scale=2.5)
    torch.cuda.synchronize()
    assert torch.equal(lg[0], lg[1]) and torch.equal(idx[0], idx[1]) and torch.equal(w[0], w[1])
    # softmax without bias, groups or factor is mok_topk's rule
    mok.mok_topk(lg[0], k, idx[0], w[0])
    mok.mok_topk_scored(lg[0], k, idx[1], w[1], score="softmax")
    torch.cuda.synchronize()
    assert torch.equal(idx[0], idx[1]) and (w[0] - w[1]).abs().max() <= 2 * U


# ------------------------------------------------------------------------------- gradient

def weights(l, idx, kind, renorm, scale):
    s = scores(l, kind)
    ok = (idx >= 0) & (idx < l.shape[1])
    p = np.where(ok, np.take_along_axis(s, np.clip(idx, 0, l.shape[1] - 1), 1), 0.0)
    if not renorm:
        return scale * p
    tot = p.sum(1, keepdims=True)
    return scale * np.where(tot > 0, p / np.where(tot > 0, tot, 1), 0)


def gradient(l, idx, dw, kind, renorm, scale):
    """d (sum w dw) / d l, and the scale its rounding goes by."""
    T, E = l.shape
    s, dw = scores(l, kind), dw.astype(np.float64)
    ok = (idx >= 0) & (idx < E)
    ix = np.clip(idx, 0, E - 1)
    p = np.where(ok, np.take_along_axis(s, ix, 1), 0.0)
    dw = np.where(ok, dw, 0.0)
    if renorm:
        tot = p.sum(1, keepdims=True)
        safe = np.where(tot > 0, tot, 1)
        dp = np.where(tot > 0, scale / safe * (dw - (dw * p).sum(1, keepdims=True) / safe), 0)
        mag = np.where(tot > 0, abs(scale) / safe * (np.abs(dw) + (np.abs(dw) * p).sum(1, keepdims=True) / safe), 0)
    else:
        dp, mag = scale * dw, np.abs(scale * dw)
    ds, m = np.zeros((T, E)), np.zeros((T, E))
    for j in range(idx.shape[1]):
        np.add.at(ds, (np.arange(T), ix[:, j]), np.where(ok[:, j], dp[:, j], 0))
        np.add.at(m, (np.arange(T), ix[:, j]), np.where(ok[:, j], mag[:, j], 0))
    if kind == "sigmoid":
        f = s * scores(-l, kind)
        return ds * f, m * f
    return (s * (ds - (ds * s).sum(1, keepdims=True)), s * (m + (m * s).sum(1, keepdims=True)))


def test_gradient_formula_against_differences():
    rng = np.random.default_rng(3)
    l = rng.standard_normal((4, 9))
    idx = np.array([[0, 3, 8], [2, 2, 5], [1, 9, 4], [7, -1, 7]])
    dw = rng.standard_normal((4, 3))
    for kind in ("sigmoid", "softmax"):
        for renorm in (True, False):
            ref, _ = gradient(l, idx, dw, kind, renorm, 1.7)
            for e in range(9):
                h = np.zeros_like(l)
                h[:, e] = 1e-6
                num = ((weights(l + h, idx, kind, renorm, 1.7) - weights(l - h, idx, kind, renorm, 1.7)) * dw).sum(1) / 2e-6
                assert np.abs(num - ref[:, e]).max() < 1e-8


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (70, 64, 6), (33, 256, 8), (9, 100, 9), (20, 384, 8),
                                   (3, 1024, 64), (300, 20, 4), (1000, 8, 2), (2, 1021, 33)])
def test_gradient(T, E, k, score, renorm):
    import routing_grouped_expert_gemm_amd as mok
    rng = np.random.default_rng(T + E)
    l, dw = logits(rng, T, E), rng.standard_normal((T, k)).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if T > 4:
        idx[0, 0] = -1                                   # takes no part
        idx[1, -1] = E + 5
        idx[2, :] = idx[2, 0]                            # one expert throughout
        idx[3, :] = -1
    din = rng.standard_normal((T, E)).astype(np.float32)
    D = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    out, out2 = torch.full((T, E), 7.0, device=DEV), D(din)
    kw = dict(score=score, renorm=renorm, scale=1.5)
    mok.mok_topk_scored_backward(D(l), D(idx), D(dw), out, **kw)
    mok.mok_topk_scored_backward(D(l), D(idx), D(dw), out2, dlogits_in=out2, **kw)
    out3 = torch.empty_like(out)
    mok.mok_topk_scored_backward(D(l), D(idx), D(dw), out3, dlogits_in=D(din), **kw)
    torch.cuda.synchronize()
    ref, mag = gradient(l, idx, dw, score, renorm, 1.5)
    assert (np.abs(out.cpu().numpy() - ref) <= 8 * U * mag + 1e-40).all()
    assert (np.abs(out2.cpu().numpy() - (ref + din)) <= 8 * U * mag + U * np.abs(ref + din) + 1e-40).all()
    assert torch.equal(out2, out3)


def test_gradient_of_rows_without_scores():
    import routing_grouped_expert_gemm_amd as mok
    l = torch.full((4, 32), -float("inf"), device=DEV)
    l[1, 3], l[2, 5] = 0.5, -1.0
    idx = torch.tensor([[0, 1], [3, 0], [0, 1], [2, 7]], dtype=torch.int32, device=DEV)
    dw = torch.ones(4, 2, device=DEV)
    dw[:, 1] = 2
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            out = torch.full_like(l, 9.0)
            mok.mok_topk_scored_backward(l, idx, dw, out, score=score, renorm=renorm)
            torch.cuda.synchronize()
            ref, _ = gradient(l.cpu().numpy(), idx.cpu().numpy(), dw.cpu().numpy(), score, renorm, 1.0)
            assert np.abs(out.cpu().numpy() - ref).max() <= 8 * U


def test_router_gradient_without_picks():
    """mok_route_backward on dlogits alone: as with picks whose gradient is zero."""
    import routing_grouped_expert_gemm_amd as mok
    for T, d, E, t in ((40, 256, 16, torch.bfloat16), (700, 2048, 64, torch.bfloat16), (50, 33, 9, torch.float32),
                       (5000, 1024, 4, torch.float32)):
        g = torch.Generator(device=DEV).manual_seed(T)
        r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        x, w, dl = r(T, d).to(t), r(E, d).to(t), r(T, E)
        ws = torch.empty(mok.mok_route_backward_workspace_bytes(T, d, E, t), dtype=torch.uint8, device=DEV)
        a = [torch.empty_like(x), torch.empty(E, d, device=DEV)]
        b = [torch.empty_like(x), torch.empty(E, d, device=DEV)]
        mok.mok_route_backward(x, w, None, None, None, *a, ws, dlogits=dl)
        idx, z = torch.zeros(T, 2, dtype=torch.int32, device=DEV), torch.zeros(T, 2, device=DEV)
        mok.mok_route_backward(x, w, idx, z, z, *b, ws, dlogits=dl)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        with pytest.raises(mok.MokError):
            mok.mok_route_backward(x, w, None, None, None, *a, ws)
        with pytest.raises(mok.MokError):
            mok.mok_route_backward(x, w, None, z, z, *a, ws, dlogits=dl)


def test_captured_and_replayed():
    """Both calls in one graph on a side stream: every replay gives the eager result of its inputs."""
    import routing_grouped_expert_gemm_amd as mok
    T, E, k = 500, 256, 8
    bias = 0.05 * torch.randn(E, device=DEV)
    l, dw = torch.randn(T, E, device=DEV), torch.randn(T, k, device=DEV)
    idx, w, dl = (torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV),
                  torch.empty(T, E, device=DEV))

    def go(i, w_, d):
        mok.mok_topk_scored(l, k, i, w_, bias=bias, n_groups=8, topk_groups=4)
        mok.mok_topk_scored_backward(l, i, dw, d)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(idx, w, dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(idx, w, dl)
    for i in range(4):
        l.normal_()
        dw.normal_()
        graph.replay()
        torch.cuda.synchronize()
        e = [torch.empty_like(v) for v in (idx, w, dl)]
        go(*e)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(e, (idx, w, dl))), i
