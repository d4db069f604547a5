"""Residual RMS norm (mok_rmsnorm, mok_rmsnorm_backward) against its definition in float64.

Tolerances, u = 2^-24. rstd comes from a sum of d squares added in chains of at most 64 values,
then in a tree: at most 80 roundings of positive terms, half of that in the square root, so y and
rstd are off by at most 64 u of themselves, and by half a step of the output type. dx is a
difference: 128 u of rstd (|g| + |n| mean|g n|) + |dh|, and half a step. dweight sums rows in
chains of at most 64 (512 workgroups, 16 groups of their shares): 128 u of sum |dy n|. The
one-value-a-step form adds chains of d / 256 values, at most 128 here: the same bounds doubled."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def half_step(t):
    return 0.0 if t is torch.float32 else torch.finfo(t).eps / 2


def inputs(T, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + d)
    t = TYPES[dtype]
    x, res = torch.randn(T, d, generator=g).to(t), (2 * torch.randn(T, d, generator=g)).to(t)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(t)
    dy, dh = torch.randn(T, d, generator=g).to(t), torch.randn(T, d, generator=g).to(t)
    return x, res, w, dy, dh


def reference(x, res, w, dy=None, dh=None, eps=EPS):
    h = x if res is None else (x.double() + res.double()).to(x.dtype)
    v, wt = h.double().numpy(), w.double().numpy()
    rstd = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    n = v * rstd
    out = dict(h=h, rstd=rstd[:, 0], y=n * wt)
    if dy is not None:
        dyv = dy.double().numpy()
        g = dyv * wt
        m = (g * n).mean(1, keepdims=True)
        o = 0.0 if dh is None else dh.double().numpy()
        out["dx"] = rstd * (g - n * m) + o
        out["dx_scale"] = rstd * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True)) \
            + np.abs(o)
        out["dw"] = (dyv * n).sum(0)
        out["dw_scale"] = np.abs(dyv * n).sum(0)
    return out


def near(got, ref, tol, t):
    got = got.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol + half_step(t) * np.abs(ref) + 1e-37).all()


SHAPES = [(1, 1), (1, 8), (3, 5), (2, 32), (5, 33), (4, 96), (9, 512), (7, 520), (6, 1000),
          (4, 1024), (5, 1160), (130, 2048), (3, 2056), (5, 4096), (3, 4100), (3, 7168), (2, 8192),
          (2, 8200), (1, 16384), (2, 16392), (1, 20000), (700, 64), (2100, 256), (530, 2304)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_against_float64(T, d, dtype):
    import routing_grouped_expert_gemm_amd as mok
    t = TYPES[dtype]
    wide = 2 if d % 8 or d > 8192 else 1
    x, res, w, dy, dh = inputs(T, d, dtype)
    ref = reference(x, res, w, dy, dh)
    D = [v.to(DEV) for v in (x, res, w, dy, dh)]
    h, y, dx = (torch.full((T, d), 7.0, dtype=t, device=DEV) for _ in range(3))
    rstd, dw = torch.full((T,), 7.0, device=DEV), torch.full((d,), 7.0, device=DEV)
    ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_rmsnorm(D[0], D[2], EPS, residual=D[1], h=h, y=y, rstd=rstd)
    mok.mok_rmsnorm_backward(D[3], h, rstd, D[2], dx, dw, ws, dh=D[4])
    torch.cuda.synchronize()
    assert torch.equal(h.cpu(), ref["h"])
    near(rstd, ref["rstd"], wide * 64 * U * ref["rstd"], torch.float32)
    near(y, ref["y"], wide * 64 * U * np.abs(ref["y"]), t)
    near(dx, ref["dx"], wide * 128 * U * ref["dx_scale"], t)
    near(dw, ref["dw"], wide * 128 * U * ref["dw_scale"], torch.float32)
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    mok.mok_rmsnorm_backward(D[3], h, rstd, D[2], dx2, dw2, ws, dh=D[4])
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    # without residual, upstream stream gradient and weight gradient
    mok.mok_rmsnorm(D[0], D[2], EPS, y=y)
    mok.mok_rmsnorm(D[0], D[2], EPS, rstd=rstd)
    mok.mok_rmsnorm_backward(D[3], D[0], rstd, D[2], dx)
    torch.cuda.synchronize()
    ref = reference(x, None, w, dy)
    near(y, ref["y"], wide * 64 * U * np.abs(ref["y"]), t)
    near(dx, ref["dx"], wide * 128 * U * ref["dx_scale"], t)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1, 32), (1, 7168), (3, 96), (4, 544), (5, 1056), (70, 2048),
                                 (3, 4128), (2, 8192), (2, 16384), (2, 16416), (1, 20000)])
def test_mxfp8_output(T, d, dtype):
    """Codes and scales are those of the norm of the stored h, rounded to float32, bit for bit: the
    library's y is off by less than 2^-44 of itself before that one rounding, so that they could
    differ only where the norm lies that close to a border of two float32 values and that one at a
    border of two codes (one value in 2^40). With float32 rows they are also the quantised y."""
    import routing_grouped_expert_gemm_amd as mok
    x, res, w, _, _ = inputs(T, d, dtype, seed=1)
    x[0, :32] = 0
    res[0, :32] = 0                                      # a block of zeros
    D = [v.to(DEV) for v in (x, res, w)]
    codes = torch.full((T, d), 0xEE, dtype=torch.uint8, device=DEV)
    scales = torch.full((T, d // 32), 0xEE, dtype=torch.uint8, device=DEV)
    y = torch.empty_like(D[0])
    h = torch.empty_like(D[0])
    mok.mok_rmsnorm(D[0], D[2], EPS, residual=D[1], h=h, y=y, codes=codes, scales=scales)
    c1, s1 = torch.empty_like(codes), torch.empty_like(scales)
    mok.mok_rmsnorm(h, D[2], EPS, codes=c1, scales=s1)
    torch.cuda.synchronize()
    assert torch.equal(c1, codes) and torch.equal(s1, scales)
    if dtype == "fp32":
        mok.mok_quantize_mxfp8_f32(y, c1, s1)
        torch.cuda.synchronize()
        assert torch.equal(c1, codes) and torch.equal(s1, scales)
    ref = reference(x, res, w)["y"].astype(np.float32).astype(np.float64).reshape(T, -1, 32)
    amax = np.abs(ref).max(2)
    exp = np.where(amax > 0, np.frexp(amax)[1] - 1 - 8, -127)
    assert np.array_equal(scales.cpu().numpy().astype(int), exp + 127)
    u = np.abs(ref) * 2.0 ** -exp[:, :, None].astype(float)
    step = 2.0 ** (np.maximum(np.frexp(u)[1] - 1, -6) - 3.0)
    val = np.minimum(np.rint(u / step) * step, 448.0)             # half to even
    got = codes.cpu().view(torch.float8_e4m3fn).double().numpy().reshape(ref.shape)
    assert np.array_equal(np.abs(got), val)
    assert np.array_equal(np.signbit(got)[val > 0], (ref < 0)[val > 0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_float32_norm_is_rounded_once(dtype):
    """y of float32 rows is the float64 norm rounded to float32: off by at most half a step and
    2^-44, so equal but where it lies within 2^-44 of the middle of two values (one in 2^20, and
    one in 65,536 is allowed). Values that bf16 holds, and any."""
    import routing_grouped_expert_gemm_amd as mok
    for T, d in ((40, 1792), (33, 7168), (9, 16384), (5, 1001)):
        x, _, w, _, _ = inputs(T, d, dtype, seed=5)
        x, w = x.float(), w.float()
        y = torch.empty(T, d, device=DEV)
        mok.mok_rmsnorm(x.to(DEV), w.to(DEV), EPS, y=y)
        torch.cuda.synchronize()
        ref = reference(x, None, w, eps=float(np.float32(EPS)))["y"].astype(np.float32)
        assert (y.cpu().numpy() != ref).sum() <= T * d >> 16


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 100, 2048, 7168, 9000])
def test_rows_at_the_ends_of_the_range(d, dtype):
    """Rows of 1e38, where h weight is past float32 though y is not; of 1e-38 and 1e-40, where (eps
    0) h weight is a subnormal or rstd past float32; one large value among small ones."""
    import routing_grouped_expert_gemm_amd as mok
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(d)
    v = torch.rand(4, d, generator=g, dtype=torch.float64) + 0.5
    v *= torch.tensor([1e38, 1e-38, 1e-40, 1.0], dtype=torch.float64)[:, None]
    v[3, d // 2] = 1e38
    x = (v * torch.where(torch.rand(4, d, generator=g) < 0.5, -1, 1)).to(t)
    w = (8 * torch.randn(d, generator=g)).to(t)
    y = torch.empty(4, d, dtype=t, device=DEV)
    mok.mok_rmsnorm(x.to(DEV), w.to(DEV), 0.0, y=y)
    ref = reference(x, None, w, eps=0.0)
    near(y, ref["y"], 2 * 64 * U * np.abs(ref["y"]), t)


def test_mxfp8_marks_what_is_not_finite():
    """A NaN or an infinity in a row: the blocks of y that hold a NaN are all NaN (0x7F, 0xFF)."""
    import routing_grouped_expert_gemm_amd as mok
    for d in (64, 8192 + 64, 16384 + 32):
        x = torch.randn(3, d, generator=torch.Generator().manual_seed(1))
        x[0, 40], x[1, 3] = float("nan"), float("inf")
        codes = torch.empty((3, d), dtype=torch.uint8, device=DEV)
        scales = torch.empty((3, d // 32), dtype=torch.uint8, device=DEV)
        mok.mok_rmsnorm(x.to(DEV), torch.ones(d, device=DEV), EPS, codes=codes, scales=scales)
        torch.cuda.synchronize()
        c, s = codes.cpu(), scales.cpu()
        assert (c[0] == 0x7F).all() and (s[0] == 0xFF).all()        # a NaN is in every value
        assert (c[1, :32] == 0x7F).all() and s[1, 0] == 0xFF        # inf * 0
        assert not (c[1, 32:] & 0x7F).any()                         # finite * 0
        assert (s[2] != 0xFF).all()


@pytest.mark.parametrize("d", [64, 1001, 16400])
def test_in_place(d):
    """h over x or residual, y over x, dx over dy or dh: as the documentation allows."""
    import routing_grouped_expert_gemm_amd as mok
    T = 5
    x, res, w, dy, dh = (v.to(DEV) for v in inputs(T, d, "bf16", seed=2))
    h, y, dx, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), \
        torch.empty(T, device=DEV)
    dw, dw2 = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_rmsnorm(x, w, EPS, residual=res, h=h, y=y, rstd=rstd)
    mok.mok_rmsnorm_backward(dy, h, rstd, w, dx, dw, ws, dh=dh)
    for over in ("x", "res"):
        a, b, y2 = x.clone(), res.clone(), torch.empty_like(x)
        mok.mok_rmsnorm(a, w, EPS, residual=b, h=a if over == "x" else b, y=y2)
        torch.cuda.synchronize()
        assert torch.equal(a if over == "x" else b, h) and torch.equal(y2, y)
    a, b = x.clone(), res.clone()
    mok.mok_rmsnorm(a, w, EPS, residual=b, h=b, y=a)
    torch.cuda.synchronize()
    assert torch.equal(b, h) and torch.equal(a, y)
    a = x.clone()
    mok.mok_rmsnorm(a, w, EPS, residual=res, y=a)
    torch.cuda.synchronize()
    assert torch.equal(a, y)
    for over in ("dy", "dh"):
        a, b = dy.clone(), dh.clone()
        mok.mok_rmsnorm_backward(a, h, rstd, w, a if over == "dy" else b, dw2, ws, dh=b)
        torch.cuda.synchronize()
        assert torch.equal(a if over == "dy" else b, dx) and torch.equal(dw2, dw)


def test_gradient_against_differences():
    """Central differences in float64 of the definition, along random directions: with step h the
    quotient is off by h^2 of the third derivative (a few units at most at this scale)."""
    import routing_grouped_expert_gemm_amd as mok
    T, d = 4, 48
    x, _, w, dy, _ = inputs(T, d, "fp32", seed=3)
    rstd, dx, dw = torch.empty(T, device=DEV), torch.empty(T, d, device=DEV), \
        torch.empty(d, device=DEV)
    ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_rmsnorm(x.to(DEV), w.to(DEV), EPS, rstd=rstd)
    mok.mok_rmsnorm_backward(dy.to(DEV), x.to(DEV), rstd, w.to(DEV), dx, dw, ws)
    torch.cuda.synchronize()

    def f(xv, wv):
        r = 1 / torch.sqrt((xv * xv).mean(1, keepdim=True) + EPS)
        return float((xv * r * wv * dy.double()).sum())

    g = torch.Generator().manual_seed(6)
    for _ in range(8):
        vx = torch.randn(T, d, generator=g, dtype=torch.float64)
        vw = torch.randn(d, generator=g, dtype=torch.float64)
        hh = 1e-4
        num = (f(x.double() + hh * vx, w.double()) - f(x.double() - hh * vx, w.double())) / (2 * hh)
        ana = float((dx.cpu().double() * vx).sum())
        assert abs(num - ana) <= 1e-4 * float((dx.cpu().double() * vx).abs().sum())
        num = (f(x.double(), w.double() + hh * vw) - f(x.double(), w.double() - hh * vw)) / (2 * hh)
        ana = float((dw.cpu().double() * vw).sum())
        assert abs(num - ana) <= 1e-4 * float((dw.cpu().double() * vw).abs().sum())


def test_no_rows():
    import routing_grouped_expert_gemm_amd as mok
    w, e = torch.ones(64, device=DEV), torch.empty((0, 64), device=DEV)
    rstd, dw = torch.empty(0, device=DEV), torch.full((64,), 7.0, device=DEV)
    ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(0, 64), dtype=torch.uint8, device=DEV)
    mok.mok_rmsnorm(e, w, EPS, y=torch.empty_like(e))
    mok.mok_rmsnorm_backward(e, e, rstd, w, torch.empty_like(e), dw, ws)
    torch.cuda.synchronize()
    assert not dw.any()


def test_rows_behind_the_last_stay():
    """Outputs longer than the rows given: what lies behind is left as it was."""
    import routing_grouped_expert_gemm_amd as mok
    for d in (64, 2304, 100):
        x = torch.randn(9, d, device=DEV)
        y = torch.full((16, d), 7.0, device=DEV)
        mok.mok_rmsnorm(x, torch.ones(d, device=DEV), EPS, y=y[:9])
        torch.cuda.synchronize()
        assert (y[9:] == 7.0).all() and torch.isfinite(y[:9]).all()


def test_graph_replays_on_another_stream():
    import routing_grouped_expert_gemm_amd as mok
    T, d = 300, 2048
    x, res, w, dy, dh = (v.to(DEV) for v in inputs(T, d, "bf16", seed=4))
    bx, bdy = torch.empty_like(x), torch.empty_like(dy)
    h, y, dx = (torch.empty_like(x) for _ in range(3))
    rstd, dw = torch.empty(T, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)

    def step(a, b, h, y, dx, rstd, dw):
        mok.mok_rmsnorm(a, w, EPS, residual=res, h=h, y=y, rstd=rstd)
        mok.mok_rmsnorm_backward(b, h, rstd, w, dx, dw, ws, dh=dh)

    bx.copy_(x)
    bdy.copy_(dy)
    step(bx, bdy, h, y, dx, rstd, dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(bx, bdy, h, y, dx, rstd, dw)
    side = torch.cuda.Stream()
    for i in range(4):
        xi, dyi = (x * (i + 1)).contiguous(), (dy * (2 - i)).contiguous()
        e = [torch.empty_like(v) for v in (h, y, dx, rstd, dw)]
        step(xi, dyi, *e)
        bx.copy_(xi)
        bdy.copy_(dyi)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(e, (h, y, dx, rstd, dw)):
            assert torch.equal(a, b)
