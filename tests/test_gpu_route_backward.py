"""Router backward (mok_route_backward) against its definition in float64.

Tolerances, u = 2^-24. dl is a sum of products formed in float32: with D = |dlogits| + the
absolute terms of the picks, its error is at most (k + 8) u D. dx adds E products of dl (kept to
16 bits at least: 2^-16 D) and the weight, dw_router T products of dl (24 bits) and x, in any order:
dx is off by ((E + k + 10) u + 2^-16) sum D |W| + u |dx|, dw_router by (T + k + 10) u sum D |x|, and
dx by half a step of its type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def inputs(T, d, E, k, dtype, seed=0):
    g = torch.Generator().manual_seed(seed * 104729 + T * 131 + d * 7 + E)
    t = TYPES[dtype]
    x = torch.randn(T, d, generator=g).to(t)
    w = (torch.randn(E, d, generator=g) * d ** -0.5).to(t)
    top = torch.topk(torch.randn(T, E, generator=g), k, dim=1)
    return dict(x=x, w=w, idx=top.indices.int(), tw=torch.softmax(top.values, 1),
                dtw=torch.randn(T, k, generator=g), dl=torch.randn(T, E, generator=g) * 0.1,
                dx_in=torch.randn(T, d, generator=g).to(t))


def reference(i, dlogits=True, dx_in=True):
    E = i["w"].shape[0]
    idx, tw, dtw = i["idx"].numpy(), i["tw"].double().numpy(), i["dtw"].double().numpy()
    ok = (idx >= 0) & (idx < E)
    tw = np.where(ok, tw, 0.0)
    s = np.where(ok, tw * dtw, 0.0).sum(1, keepdims=True)
    g, ga = np.where(ok, tw * (dtw - s), 0.0), np.where(ok, tw * (np.abs(dtw) + np.abs(tw * dtw).sum(1, keepdims=True)), 0.0)
    dl = i["dl"].double().numpy().copy() if dlogits else np.zeros(i["dl"].shape)
    D = np.abs(dl)
    rows = np.arange(idx.shape[0])
    for j in range(idx.shape[1]):
        e = np.where(ok[:, j], idx[:, j], 0)
        np.add.at(dl, (rows, e), g[:, j])
        np.add.at(D, (rows, e), ga[:, j])
    x, w = i["x"].double().numpy(), i["w"].double().numpy()
    o = i["dx_in"].double().numpy() if dx_in else 0.0
    return dict(dx=dl @ w + o, dxs=D @ np.abs(w), dw=dl.T @ x, dws=D.T @ np.abs(x))


def run(mok, i, dlogits=True, dx_in=True, want=("dx", "dw")):
    x, w = i["x"].to(DEV), i["w"].to(DEV)
    (T, d), E = x.shape, w.shape[0]
    dx = torch.full_like(x, 7.0) if "dx" in want else None
    dw = torch.full((E, d), 7.0, device=DEV) if "dw" in want else None
    ws = torch.full((mok.mok_route_backward_workspace_bytes(T, d, E, x.dtype),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    mok.mok_route_backward(x, w, i["idx"].to(DEV), i["tw"].to(DEV), i["dtw"].to(DEV), dx, dw, ws,
                           dlogits=i["dl"].to(DEV) if dlogits else None,
                           dx_in=i["dx_in"].to(DEV) if dx_in else None)
    torch.cuda.synchronize()
    return dx, dw


def check(dx, dw, ref, T, E, k, t):
    half = 0.0 if t is torch.float32 else torch.finfo(t).eps / 2
    if dx is not None:
        got = dx.double().cpu().numpy()
        tol = ((E + k + 10) * U + 2.0 ** -16) * ref["dxs"] + (U + half) * np.abs(ref["dx"]) * 1.01
        assert (np.abs(got - ref["dx"]) <= tol + half * ref["dxs"] * 2.0 ** -15).all()
    if dw is not None:
        got = dw.double().cpu().numpy()
        assert (np.abs(got - ref["dw"]) <= (T + k + 10) * U * ref["dws"]).all()


CASES = [  # T, d, E, k
    (1, 1, 1, 1), (1, 64, 8, 2), (3, 17, 5, 5), (45, 144, 16, 4), (257, 272, 20, 4), (64, 128, 64, 6),
    (100, 100, 63, 3), (130, 192, 65, 8), (33, 256, 96, 8), (300, 448, 130, 8), (70, 512, 256, 8),
    (129, 320, 384, 8), (31, 64, 1000, 16), (20, 128, 1024, 64), (1000, 2048, 64, 6),
    (2100, 64, 16, 2), (5000, 40, 8, 2), (512, 2056, 64, 6), (515, 1984, 32, 4), (700, 1999, 130, 8), (40, 30001, 128, 4)]


# enough tiles for the wide form of bf16: 768 of 128 tokens x 256 columns
WIDE = [(16500, 1416, 20, 4), (16400, 1288, 130, 8), (98300, 8, 64, 6), (256, 98056, 100, 8),
        (1024, 24584, 257, 8),
        # rows that are copied to 16 bytes: 2^25 products or more of another d than whole pieces
        (16500, 1417, 20, 4), (16400, 1283, 130, 8), (98300, 11, 64, 6), (5536, 1069, 212, 6),
        (1030, 1020, 64, 6), (2100, 2047, 16, 2), (33000, 3, 1000, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d,E,k", CASES)
def test_against_float64(T, d, E, k, dtype):
    import routing_grouped_expert_gemm_amd as mok
    i = inputs(T, d, E, k, dtype)
    dx, dw = run(mok, i)
    check(dx, dw, reference(i), T, E, k, TYPES[dtype])
    dx2, dw2 = run(mok, i)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d,E,k", [(2100, 2003, 7, 3), (70000, 61, 5, 5), (4200, 1000, 8, 8),
                                     (65, 65539, 4, 2), (4195000, 1, 1, 1), (1100, 4001, 16, 4),
                                     (4100, 1030, 1, 1)])
def test_few_experts(T, d, E, k, dtype):
    import routing_grouped_expert_gemm_amd as mok
    i = inputs(T, d, E, k, dtype)
    dx, dw = run(mok, i)
    check(dx, dw, reference(i), T, E, k, TYPES[dtype])
    for want in ("dx", "dw"):
        a, b = run(mok, i, want=(want,))
        assert torch.equal(a, dx) if want == "dx" else torch.equal(b, dw)
    dx, dw = run(mok, i, False, False)
    check(dx, dw, reference(i, False, False), T, E, k, TYPES[dtype])


@pytest.mark.parametrize("T,d,E,k", WIDE)
def test_wide_against_float64(T, d, E, k):
    import routing_grouped_expert_gemm_amd as mok
    i = inputs(T, d, E, k, "bf16")
    dx, dw = run(mok, i)
    check(dx, dw, reference(i), T, E, k, torch.bfloat16)
    for want in ("dx", "dw"):                 # either product alone: the same bits
        a, b = run(mok, i, want=(want,))
        assert torch.equal(a, dx) if want == "dx" else torch.equal(b, dw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_optional_parts(dtype):
    import routing_grouped_expert_gemm_amd as mok
    T, d, E, k = 150, 192, 64, 6
    i = inputs(T, d, E, k, dtype, seed=1)
    for dl in (True, False):
        for dxi in (True, False):
            ref = reference(i, dl, dxi)
            dx, dw = run(mok, i, dl, dxi)
            check(dx, dw, ref, T, E, k, TYPES[dtype])
            one, none = run(mok, i, dl, dxi, want=("dx",))
            assert none is None and torch.equal(one, dx)
            none, one = run(mok, i, dl, dxi, want=("dw",))
            assert none is None and torch.equal(one, dw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_picks_outside_and_repeated(dtype):
    import routing_grouped_expert_gemm_amd as mok
    T, d, E, k = 100, 128, 64, 4
    i = inputs(T, d, E, k, dtype, seed=2)
    i["idx"][3] = torch.tensor([5, 5, 5, 9])
    i["idx"][4] = torch.tensor([-1, E, 2 ** 31 - 1, 7])
    i["idx"][5] = -(2 ** 31)
    dx, dw = run(mok, i)
    check(dx, dw, reference(i), T, E, k, TYPES[dtype])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 50), ("bf16", 13625), ("fp32", 64),
                                     ("fp32", 54473)])
def test_dx_over_dx_in_and_rows_behind(dtype, d):
    import routing_grouped_expert_gemm_amd as mok
    T, E, k = 77, 64, 6
    i = inputs(T, d, E, k, dtype, seed=3)
    dx, dw = run(mok, i)
    buf = torch.full((T + 9, d), 7.0, dtype=TYPES[dtype], device=DEV)
    buf[:T] = i["dx_in"].to(DEV)
    dw2 = torch.empty_like(dw)
    ws = torch.empty(mok.mok_route_backward_workspace_bytes(T, d, E, TYPES[dtype]),
                     dtype=torch.uint8, device=DEV)
    mok.mok_route_backward(i["x"].to(DEV), i["w"].to(DEV), i["idx"].to(DEV), i["tw"].to(DEV),
                           i["dtw"].to(DEV), buf[:T], dw2, ws, dlogits=i["dl"].to(DEV),
                           dx_in=buf[:T])
    torch.cuda.synchronize()
    assert torch.equal(buf[:T], dx) and torch.equal(dw2, dw) and (buf[T:] == 7.0).all()


def test_no_tokens():
    import routing_grouped_expert_gemm_amd as mok
    i = inputs(0, 64, 8, 2, "bf16")
    dx, dw = run(mok, i)
    assert dx.shape == (0, 64) and not dw.any()


def test_gradient_against_differences():
    """Directional central differences in float64 of sum(topk_w v) + sum(logits c) through the
    router's definition, picks fixed; the quotient's own error is h^2 of a third derivative."""
    import routing_grouped_expert_gemm_amd as mok
    T, d, E, k = 6, 32, 10, 3
    i = inputs(T, d, E, k, "fp32", seed=4)
    lg = i["x"].double() @ i["w"].double().T
    top = torch.topk(lg, k, dim=1)
    i["idx"], i["tw"] = top.indices.int(), torch.softmax(top.values, 1).float()
    dx, dw = run(mok, i, dx_in=False)

    def f(x, w):
        lg = x @ w.T
        tw = torch.softmax(torch.gather(lg, 1, i["idx"].long()), 1)
        return float((tw * i["dtw"].double()).sum() + (lg * i["dl"].double()).sum())

    g = torch.Generator().manual_seed(8)
    for _ in range(6):
        vx = torch.randn(T, d, generator=g, dtype=torch.float64)
        vw = torch.randn(E, d, generator=g, dtype=torch.float64)
        x, w, h = i["x"].double(), i["w"].double(), 1e-4
        num = (f(x + h * vx, w) - f(x - h * vx, w)) / (2 * h)
        part = dx.cpu().double() * vx
        assert abs(num - float(part.sum())) <= 1e-4 * float(part.abs().sum())
        num = (f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h)
        part = dw.cpu().double() * vw
        assert abs(num - float(part.sum())) <= 1e-4 * float(part.abs().sum())


@pytest.mark.parametrize("dtype,T,d,E", [("bf16", 90, 64, 32), ("bf16", 1100, 1001, 64),
                                         ("bf16", 1100, 1024, 64), ("fp32", 90, 64, 32)])
def test_any_address(dtype, T, d, E):
    """Tensors that start one value behind a 16-byte address."""
    import routing_grouped_expert_gemm_amd as mok
    k = 5
    i = inputs(T, d, E, k, dtype, seed=6)

    def off(v):
        b = torch.empty(v.numel() + 1, dtype=v.dtype, device=DEV)
        b[1:] = v.to(DEV).flatten()
        return b[1:].view(v.shape)

    dx, dw = off(torch.full((T, d), 7.0).to(TYPES[dtype])), off(torch.full((E, d), 7.0))
    ws = torch.empty(mok.mok_route_backward_workspace_bytes(T, d, E, TYPES[dtype]),
                     dtype=torch.uint8, device=DEV)
    mok.mok_route_backward(off(i["x"]), off(i["w"]), off(i["idx"]), off(i["tw"]), off(i["dtw"]), dx,
                           dw, ws, dlogits=off(i["dl"]), dx_in=off(i["dx_in"]))
    torch.cuda.synchronize()
    check(dx, dw, reference(i), T, E, k, TYPES[dtype])


@pytest.mark.parametrize("d", [256, 100, 1003])
def test_graph_replays(d):
    import routing_grouped_expert_gemm_amd as mok
    T, E, k = 1100, 64, 6
    dev = {n: v.to(DEV) for n, v in inputs(T, d, E, k, "bf16", seed=5).items()}
    x, dl = dev["x"].clone(), dev["dl"].clone()
    dx, dw = torch.empty_like(x), torch.empty(E, d, device=DEV)
    ws = torch.empty(mok.mok_route_backward_workspace_bytes(T, d, E, x.dtype), dtype=torch.uint8,
                     device=DEV)

    def step(x, dl, dx, dw):
        mok.mok_route_backward(x, dev["w"], dev["idx"], dev["tw"], dev["dtw"], dx, dw, ws,
                               dlogits=dl, dx_in=dev["dx_in"])

    step(x, dl, dx, dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, dl, dx, dw)
    for n in range(4):
        xi, dli = (dev["x"] * (n + 1)).contiguous(), (dev["dl"] * (n - 2)).contiguous()
        e = torch.empty_like(dx), torch.empty_like(dw)
        step(xi, dli, *e)
        x.copy_(xi)
        dl.copy_(dli)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(e[0], dx) and torch.equal(e[1], dw)
