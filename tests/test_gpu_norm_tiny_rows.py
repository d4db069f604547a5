"""Backward of the residual RMS norm with eps 0 for rows whose rstd no float32 holds: root mean
squares below 3e-39. Their norm is an ordinary number, so dweight is one too, and dx is where dy is
small enough.

Tolerances: those of the norm's tests, u = 2^-24: 128 u of the absolute terms (256 u in the form of
one value a step), half a step of the type, and half a step of float32's subnormals."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def reference(h, w, dy, dh):
    v, wt, g0 = (t.double().numpy() for t in (h, w, dy))
    rstd = 1 / np.sqrt((v * v).mean(1, keepdims=True))
    n, g = v * rstd, g0 * wt
    gn = (g * n).mean(1, keepdims=True)
    o = 0.0 if dh is None else dh.double().numpy()
    return dict(rstd=rstd[:, 0], dx=rstd * (g - n * gn) + o,
                dx_scale=rstd * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True)) + np.abs(o),
                dw=(g0 * n).sum(0), dw_scale=np.abs(g0 * n).sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("d", [1, 64, 100, 512, 1024, 2048, 4096, 7168, 9000])
def test_backward_of_rows_below_float32s_rstd(d, T, dtype):
    import routing_grouped_expert_gemm_amd as mok
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(d + T)
    v = (torch.rand(T, d, generator=g, dtype=torch.float64) + 0.5) * 1e-40
    v[1::2] *= 1e40                                        # every other row an ordinary one
    if T > 4:
        v[4] *= 20                                         # rms about 2e-39
    x = (v * torch.where(torch.rand(T, d, generator=g) < 0.5, -1, 1)).to(t)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(t)
    dy, dh = torch.randn(T, d, generator=g).to(t), torch.randn(T, d, generator=g).to(t)
    ref = reference(x, w, dy, None)
    small = torch.where(torch.arange(T) % 2 == 0, 2.0 ** -40, 1.0)[:, None]   # keeps dx inside float32
    for scale, with_dh in ((1.0, False), (small, False), (small, True)):
        dys = (dy * scale).to(t)
        ref = reference(x, w, dys, dh if with_dh else None)
        D = [u.to(DEV) for u in (x, w, dys, dh)]
        rstd, dw = torch.empty(T, device=DEV), torch.full((d,), 7.0, device=DEV)
        dx = torch.empty(T, d, dtype=t, device=DEV)
        ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
        mok.mok_rmsnorm(D[0], D[1], 0.0, rstd=rstd)
        mok.mok_rmsnorm_backward(D[2], D[0], rstd, D[1], dx, dw, ws, dh=D[3] if with_dh else None)
        torch.cuda.synchronize()
        assert torch.isinf(rstd[0::2]).all() and torch.isfinite(rstd[1::2]).all()
        wide = 2 if d % 8 else 1
        got = dw.double().cpu().numpy()
        assert (np.abs(got - ref["dw"]) <= wide * 128 * U * ref["dw_scale"]).all()
        fits = np.abs(ref["dx"]) + ref["dx_scale"] < 1e38
        assert fits[1::2].all() and (with_dh is False or fits.all())
        got = dx.double().cpu().numpy()
        half = 0.0 if t is torch.float32 else torch.finfo(t).eps / 2
        tol = wide * 128 * U * ref["dx_scale"] + half * np.abs(ref["dx"]) + 2.0 ** -134
        with np.errstate(invalid="ignore"):                # infinities where dx is past float32
            assert (np.abs(got - ref["dx"]) <= tol)[fits].all()
        assert not np.isnan(got).any()


def test_rows_in_place_and_replayed():
    """dx over dy, and a captured call that meets such rows only in some replays."""
    import routing_grouped_expert_gemm_amd as mok
    T, d = 40, 1024
    h = torch.randn(T, d, device=DEV)
    w, dy, rstd = torch.ones(d, device=DEV), torch.randn(T, d, device=DEV), torch.ones(T, device=DEV)
    dx, dw = torch.empty_like(h), torch.empty(d, device=DEV)
    ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_rmsnorm_backward(dy, h, rstd, w, dx, dw, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mok.mok_rmsnorm(h, w, 0.0, rstd=rstd)
        mok.mok_rmsnorm_backward(dy, h, rstd, w, dx, dw, ws)
    for n in range(4):
        h.copy_(torch.randn(T, d, device=DEV))
        if n % 2:
            h[3::5] *= 1e-40
        graph.replay()
        torch.cuda.synchronize()
        assert bool(torch.isinf(rstd[3])) == bool(n % 2) and torch.isfinite(dw).all()
        e, ew = dy.clone(), torch.empty_like(dw)
        mok.mok_rmsnorm_backward(e, h, rstd, w, e, ew, ws)
        torch.cuda.synchronize()
        assert torch.equal(e, dx) and torch.equal(ew, dw)
