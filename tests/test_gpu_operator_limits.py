"""Calls of the operators around the layer that the documentation allows and that address far: tensors
past 2^31 elements, one workspace shared by two captured graphs, calls on two streams at once."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def test_norm_past_2_31_elements():
    """The last rows' results are those of a call on these rows alone."""
    import routing_grouped_expert_gemm_amd as mok
    T, d, tail = 300_100, 7200, 50
    x = torch.zeros(T, d, dtype=BF, device=DEV)
    x[-tail:] = torch.randn(tail, d, device=DEV).to(BF)
    w = torch.ones(d, dtype=BF, device=DEV)
    y, codes = torch.empty_like(x), torch.empty(T, d, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, d // 32, dtype=torch.uint8, device=DEV)
    rstd = torch.empty(T, device=DEV)
    mok.mok_rmsnorm(x, w, 1e-6, y=y, rstd=rstd, codes=codes, scales=scales)
    xs = x[-tail:].clone()
    ys, cs, ss, rs = (torch.empty_like(t[-tail:]) for t in (y, codes, scales, rstd))
    mok.mok_rmsnorm(xs, w, 1e-6, y=ys, rstd=rs, codes=cs, scales=ss)
    torch.cuda.synchronize()
    for a, b in ((y, ys), (codes, cs), (scales, ss), (rstd, rs)):
        assert torch.equal(a[-tail:], b)
    dx, dw, dws = torch.empty_like(x), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_rmsnorm_backward(y, x, rstd, w, dx, dw, ws)
    dxs = torch.empty_like(ys)
    mok.mok_rmsnorm_backward(ys, xs, rs, w, dxs, dws, ws)
    torch.cuda.synchronize()
    assert torch.equal(dx[-tail:], dxs)
    # the other rows are zero: the same 50 terms, in another order (at most 50 roundings)
    assert (dw - dws).abs().max() <= 50 * 2.0 ** -24 * (ys.float() * xs.float() * rs[:, None]).abs().sum(0).max()


def test_balance_past_2_31_elements():
    """Two sequences, the second one the last 100 tokens: its results are those of a call in which
    only these tokens exist."""
    import routing_grouped_expert_gemm_amd as mok
    E, k, tail = 1024, 8, 100
    T = (1 << 21) + 77
    logits = torch.zeros(T, E, device=DEV)
    logits[-tail:] = torch.randn(tail, E, device=DEV)
    idx = torch.randint(0, E, (T, k), dtype=torch.int32, device=DEV)

    def run(lg, ix, off):
        n = len(off) - 1
        so = torch.tensor(off, dtype=torch.int32, device=DEV)
        loss, counts = torch.empty(1, device=DEV), torch.empty(n, E, dtype=torch.int32, device=DEV)
        mean, dl = torch.empty(n, E, device=DEV), torch.empty_like(lg)
        ws = torch.empty(mok.mok_balance_loss_workspace_bytes(lg.shape[0], E, n), dtype=torch.uint8,
                         device=DEV)
        mok.mok_balance_loss(lg, ix, 1.0, loss, counts, mean, ws, seq_offsets=so)
        mok.mok_balance_loss_backward(lg, counts, k, 1.0, torch.ones(1, device=DEV), dl,
                                      seq_offsets=so)
        torch.cuda.synchronize()
        return counts, mean, dl

    c, m, dl = run(logits, idx, [0, T - tail, T])
    cs, ms, dls = run(logits[-tail:].clone(), idx[-tail:].clone(), [0, 0, tail])
    assert torch.equal(c[1], cs[1]) and torch.equal(dl[-tail:], dls)
    # sums of 100 positive terms in other chunks
    assert ((m[1] - ms[1]).abs() <= 100 * 2.0 ** -24 * ms[1]).all()
    assert int(c.sum()) == T * k and bool((m[0] == 1.0 / E).all())


@pytest.mark.parametrize("d", [7176, 7175])
def test_route_backward_past_2_31_elements(d):
    import routing_grouped_expert_gemm_amd as mok
    T, E, k, tail = 300_050, 8, 2, 60
    x = torch.zeros(T, d, dtype=BF, device=DEV)
    x[-tail:] = torch.randn(tail, d, device=DEV).to(BF)
    w = torch.randn(E, d, device=DEV).to(BF)
    idx = torch.stack([torch.randperm(E, device=DEV)[:k] for _ in range(64)]).int().repeat(
        T // 64 + 1, 1)[:T].contiguous()
    tw, dtw = torch.full((T, k), 0.5, device=DEV), torch.randn(T, k, device=DEV)

    def run(x, idx, tw, dtw):
        dx, dw = torch.empty_like(x), torch.empty(E, d, device=DEV)
        ws = torch.empty(mok.mok_route_backward_workspace_bytes(x.shape[0], d, E, BF),
                         dtype=torch.uint8, device=DEV)
        mok.mok_route_backward(x, w, idx, tw, dtw, dx, dw, ws)
        torch.cuda.synchronize()
        return dx, dw

    dx, dw = run(x, idx, tw, dtw)
    last = [t[-tail:].clone() for t in (x, idx, tw, dtw)]
    dxs, dws = run(*last)
    # dx is one row's sum over 8 experts; dw sums 60 tokens' terms in another order
    assert (dx[-tail:].float() - dxs.float()).abs().max() <= 2.0 ** -8 * dxs.float().abs().max()
    bound = 64 * 2.0 ** -24 * 2 * dtw.abs().max() * last[0].float().abs().sum(0)
    assert ((dw - dws).abs() <= bound).all()


def test_product_past_2_31_elements():
    import routing_grouped_expert_gemm_amd as mok
    M, N, K = 50_000, 50_000, 32
    rng = np.random.default_rng(0)
    u8 = lambda *s: torch.from_numpy(rng.integers(0, 256, s).astype(np.uint8)).to(DEV)  # noqa: E731
    a, b = u8(M, K // 2), u8(N, K // 2)
    sa, sb = (torch.full((n, 1), 127, dtype=torch.uint8, device=DEV) for n in (M, N))
    c = torch.empty(M, N, dtype=BF, device=DEV)
    assert mok.mok_mx_gemm_workspace_bytes(M, N, K) == 0
    mok.mok_mx_gemm(a, sa, b, sb, c)
    cs = torch.empty(40, N, dtype=BF, device=DEV)
    mok.mok_mx_gemm(a[-40:].clone(), sa[-40:].clone(), b, sb, cs)
    torch.cuda.synchronize()
    assert torch.equal(c[-40:], cs)                  # 32 products of small integers / 4: exact


def test_two_graphs_share_a_workspace():
    """Captured apart on the same workspaces, replayed one after the other in both orders."""
    import routing_grouped_expert_gemm_amd as mok
    T, E, k, d, M, N, K = 3000, 64, 6, 256, 200, 256, 8192
    made = []
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    for s in range(2):
        g = torch.Generator(device=DEV).manual_seed(s)
        lg = torch.randn(T, E, generator=g, device=DEV)
        top = torch.topk(lg, k, dim=1)
        ix, tw = top.indices.int().contiguous(), torch.softmax(top.values, 1).contiguous()
        x, w = torch.randn(T, d, generator=g, device=DEV).to(BF), torch.randn(E, d, generator=g, device=DEV).to(BF)
        dt, wn = torch.randn(T, k, generator=g, device=DEV), torch.ones(d, device=DEV).to(BF)
        qa, qb = (torch.randint(0, 256, (n, K // 2), generator=g, device=DEV, dtype=torch.uint8) for n in (M, N))
        sa, sb = (torch.randint(120, 130, (n, K // 32), generator=g, device=DEV, dtype=torch.uint8) for n in (M, N))
        o = dict(loss=torch.empty(1, device=DEV), counts=torch.empty(1, E, dtype=torch.int32, device=DEV),
                 mean=torch.empty(1, E, device=DEV), dx=torch.empty_like(x), dw=torch.empty(E, d, device=DEV),
                 dn=torch.empty_like(x), dwn=torch.empty(d, device=DEV), c=torch.empty(M, N, device=DEV))
        rstd = torch.ones(T, device=DEV)

        def step(o=o, lg=lg, ix=ix, tw=tw, dt=dt, x=x, w=w, wn=wn, qa=qa, qb=qb, sa=sa, sb=sb, rstd=rstd):
            mok.mok_balance_loss(lg, ix, 1.0, o["loss"], o["counts"], o["mean"], ws)
            mok.mok_route_backward(x, w, ix, tw, dt, o["dx"], o["dw"], ws)
            mok.mok_rmsnorm_backward(x, x, rstd, wn, o["dn"], o["dwn"], ws)
            mok.mok_mx_gemm(qa, sa, qb, sb, o["c"], ws)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        made.append((graph, o, {n: t.clone() for n, t in o.items()}, step))
    assert mok.mok_mx_gemm_workspace_bytes(M, N, K) > 0
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for i in order:
            for t in made[i][1].values():
                t.zero_()
        for i in order:
            made[i][0].replay()
        torch.cuda.synchronize()
        for i in order:
            for n, t in made[i][1].items():
                assert torch.equal(t, made[i][2][n]), n
        made[order[0]][3]()                          # eager work between the replays
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """The same calls on two streams with workspaces of their own give what one stream gives."""
    import routing_grouped_expert_gemm_amd as mok
    T, E, k, d = 20000, 64, 6, 512
    lg = torch.randn(T, E, device=DEV)
    top = torch.topk(lg, k, dim=1)
    ix, tw = top.indices.int().contiguous(), torch.softmax(top.values, 1).contiguous()
    x, w, dt = torch.randn(T, d, device=DEV).to(BF), torch.randn(E, d, device=DEV).to(BF), torch.randn(T, k, device=DEV)

    def outs():
        return (torch.empty(1, device=DEV), torch.empty(1, E, dtype=torch.int32, device=DEV),
                torch.empty(1, E, device=DEV), torch.empty_like(x), torch.empty(E, d, device=DEV))

    def calls(o, w1, w2, s):
        for _ in range(5):
            mok.mok_balance_loss(lg, ix, 1.0, o[0], o[1], o[2], w1, stream=s)
            mok.mok_route_backward(x, w, ix, tw, dt, o[3], o[4], w2, stream=s)

    n1 = mok.mok_balance_loss_workspace_bytes(T, E)
    n2 = mok.mok_route_backward_workspace_bytes(T, d, E, BF)
    scratch = [[torch.empty(n, dtype=torch.uint8, device=DEV) for n in (n1, n2)] for _ in range(3)]
    ref = outs()
    calls(ref, *scratch[0], None)
    streams, got = [torch.cuda.Stream() for _ in range(2)], [outs(), outs()]
    torch.cuda.synchronize()
    for s, o, ws in zip(streams, got, scratch[1:]):
        calls(o, *ws, s)
    torch.cuda.synchronize()
    for o in got:
        for a, b in zip(ref, o):
            assert torch.equal(a, b)
