"""Gated norm (mok_gated_norm, mok_gated_norm_backward) against its definition in float64.

Tolerances, u = 2^-24. Statistics are float64, so rstd is off by its rounding, 1 u (2 u with the
square root's), and u_i = y rstd w by 2 u. h: gate u, beta (gate u) and alpha residual are rounded
once each, their sum once: 6 u (|alpha residual| + |beta gate u|), and half a step of the storage
type. n: 4 u of itself and half a step.

The backward reads the stored rstd (1 u). nh and g take 2 roundings, mean(g nh) a chain of at most 64
values and a tree: 80 u of mean |g nh|, so dt is off by 128 u of its scale D = |dh| + rstd (|g| + |nh|
mean |g nh|). dres, dgate and q multiply by 4 roundings more: 136 u D with the factor's size. dy: p is
off by 136 u D |beta gate w|, v by 2 u, the mean by 80 u and its terms' error: 512 u of rstd (P + |v| mean
(P |v|)), P = D |beta gate w|. The sums over rows add chains of at most 64 rows and a tree: 256 u of the
sum of their terms' scales. The one-value-a-step form adds chains of d / 256 values, at most 128 here:
the same bounds doubled."""
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


def inputs(T, d, dtype, gate, post, pre, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + d)
    t = TYPES[dtype]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(y=(0.5 * r(T, d)).to(t), res=(2 * r(T, d)).to(t),
                w_post=(1 + 0.2 * r(d)).to(t) if post else None,
                w_pre=(1 + 0.2 * r(d)).to(t) if pre else None,
                gate=None if gate == "none" else r(*((T, d) if gate == "row" else (d,))).to(t),
                dh=r(T, d).to(t), dn=r(T, d).to(t) if pre else None)


def num(v):
    return None if v is None else v.double().cpu().numpy()


def rstd_of(v, eps):
    return 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def forward(a, alpha, beta, eps=EPS, h=None):
    """h before it is stored, and, from the stored h given, n."""
    y, res = num(a["y"]), num(a["res"])
    gate = 1.0 if a["gate"] is None else num(a["gate"])
    out = {}
    u = y
    if a["w_post"] is not None:
        out["rstd_y"] = rstd_of(y, eps)
        u = y * out["rstd_y"] * num(a["w_post"])
    out["h"] = alpha * res + beta * gate * u
    out["h_scale"] = np.abs(alpha * res) + np.abs(beta * gate * u)
    if h is not None and a["w_pre"] is not None:
        hv = num(h)
        out["rstd_h"] = rstd_of(hv, eps)
        out["n"] = hv * out["rstd_h"] * num(a["w_pre"])
    return out


def backward(a, h, alpha, beta, dh=True, dn=True, eps=EPS):
    y = num(a["y"])
    T, d = y.shape
    gate = np.ones((T, d)) if a["gate"] is None else np.broadcast_to(num(a["gate"]), (T, d))
    dt = num(a["dh"]) if dh else np.zeros((T, d))
    D = np.abs(dt)
    out, sc = {}, {}
    if dn and a["dn"] is not None:
        hv, g = num(h), num(a["dn"]) * num(a["w_pre"])
        r = rstd_of(hv, eps)
        nh = hv * r
        dt = dt + r * (g - nh * (g * nh).mean(1, keepdims=True))
        D = D + r * (np.abs(g) + np.abs(nh) * np.abs(g * nh).mean(1, keepdims=True))
        out["dw_pre"], sc["dw_pre"] = (num(a["dn"]) * nh).sum(0), np.abs(num(a["dn"]) * nh).sum(0)
    out["dres"], sc["dres"] = alpha * dt, np.abs(alpha) * D
    w = 1.0 if a["w_post"] is None else num(a["w_post"])
    r = 1.0 if a["w_post"] is None else rstd_of(y, eps)
    v = y * r
    dg, dgs = beta * dt * v * w, np.abs(beta * v * w) * D
    out["dgate"], sc["dgate"] = dg, dgs
    out["dgate_all"], sc["dgate_all"] = dg.sum(0), dgs.sum(0)
    q, Q = beta * dt * gate, np.abs(beta * gate) * D
    if a["w_post"] is None:
        out["dy"], sc["dy"] = q, Q
    else:
        out["dw_post"], sc["dw_post"] = (q * v).sum(0), (Q * np.abs(v)).sum(0)
        p, P = q * w, Q * np.abs(w)
        out["dy"] = r * (p - v * (p * v).mean(1, keepdims=True))
        sc["dy"] = r * (P + np.abs(v) * (P * np.abs(v)).mean(1, keepdims=True))
    return out, sc


def near(got, ref, tol, t, what=""):
    got = num(got)
    off = np.abs(got - ref) - (tol + half_step(t) * np.abs(ref) + 1e-37)
    assert (off <= 0).all(), (what, off.max())


def call(mok, D, T, d, t, alpha, beta, eps=EPS, dh=True, dn=True):
    """Both directions with everything wanted."""
    f32 = dict(device=DEV)
    post, pre, gate = (D[n] is not None for n in ("w_post", "w_pre", "gate"))
    per = gate and D["gate"].dim() == 2
    o = dict(h=torch.full((T, d), 7.0, dtype=t, device=DEV))
    o["n"] = torch.full_like(o["h"], 7.0) if pre else None
    o["rstd_y"] = torch.full((T,), 7.0, **f32) if post else None
    o["rstd_h"] = torch.full((T,), 7.0, **f32) if pre else None
    mok.mok_gated_norm(D["y"], D["res"], eps, o["h"], w_post=D["w_post"], gate=D["gate"], w_pre=D["w_pre"], n=o["n"],
                       rstd_y=o["rstd_y"], rstd_h=o["rstd_h"], alpha=alpha, beta=beta)
    o["dres"], o["dy"] = (torch.full((T, d), 7.0, dtype=t, device=DEV) for _ in range(2))
    o["dgate"] = None if not gate else torch.full((T, d), 7.0, dtype=t, device=DEV) if per else torch.full((d,), 7.0, **f32)
    o["dw_post"] = torch.full((d,), 7.0, **f32) if post else None
    o["dw_pre"] = torch.full((d,), 7.0, **f32) if pre else None
    ws = torch.empty(mok.mok_gated_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_gated_norm_backward(D["dh"] if dh else None, D["y"], o["dres"], o["dy"], ws, dn=D["dn"] if dn else None,
                                h=o["h"], gate=D["gate"], w_post=D["w_post"], w_pre=D["w_pre"], rstd_y=o["rstd_y"],
                                rstd_h=o["rstd_h"], dgate=o["dgate"], dw_post=o["dw_post"], dw_pre=o["dw_pre"],
                                alpha=alpha, beta=beta)
    torch.cuda.synchronize()
    return o


def compare(a, o, t, wide, alpha, beta, eps=EPS, dh=True, dn=True):
    f = forward(a, alpha, beta, eps, o["h"])
    near(o["h"], f["h"], wide * 6 * U * f["h_scale"], t, "h")
    for k in ("rstd_y", "rstd_h"):
        if o[k] is not None:
            near(o[k], f[k][:, 0], 2 * U * f[k][:, 0], torch.float32, k)
    if o["n"] is not None:
        near(o["n"], f["n"], 4 * U * np.abs(f["n"]), t, "n")
    b, s = backward(a, o["h"], alpha, beta, dh, dn, eps)
    near(o["dres"], b["dres"], wide * 136 * U * s["dres"], t, "dres")
    near(o["dy"], b["dy"], wide * 512 * U * s["dy"], t, "dy")
    if o["dgate"] is not None:
        if o["dgate"].dim() == 2:
            near(o["dgate"], b["dgate"], wide * 136 * U * s["dgate"], t, "dgate")
        else:
            near(o["dgate"], b["dgate_all"], wide * 256 * U * s["dgate_all"], torch.float32, "dgate")
    for k in ("dw_post", "dw_pre"):
        if o[k] is not None:
            if k in b:
                near(o[k], b[k], wide * 256 * U * s[k], torch.float32, k)
            else:
                assert (o[k] == 0).all()


SHAPES = [(1, 1), (1, 8), (3, 5), (5, 33), (9, 512), (7, 520), (6, 1000), (4, 1024), (5, 1160), (300, 1160),
          (130, 2048), (300, 2048), (3, 2056), (5, 4096), (300, 2304), (3, 4100), (3, 7168), (2, 8192), (300, 5120),
          (2, 8200), (1, 16384), (2, 16392), (700, 64), (2100, 256), (530, 111)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_against_float64(T, d, dtype):
    import routing_grouped_expert_gemm_amd as mok
    t = TYPES[dtype]
    wide = 2 if d % 8 or d > 8192 else 1
    for i, (gate, post, pre) in enumerate([("row", True, True), ("all", True, True), ("none", True, True),
                                           ("row", False, True), ("all", True, False), ("none", False, False),
                                           ("all", False, True), ("none", False, True)]):
        if T * d > 300000 and i > 2:
            break
        a = inputs(T, d, dtype, gate, post, pre)
        D = {k: None if v is None else v.to(DEV) for k, v in a.items()}
        o = call(mok, D, T, d, t, 0.875, -0.7)
        compare(a, o, t, wide, np.float32(0.875), np.float32(-0.7))
        o2 = call(mok, D, T, d, t, 0.875, -0.7)
        for k in o:
            assert o[k] is None or torch.equal(o[k], o2[k]), k
        # half of the upstream gradients
        if pre:
            compare(a, call(mok, D, T, d, t, 1.0, 1.0, dh=False), t, wide, 1.0, 1.0, dh=False)
            compare(a, call(mok, D, T, d, t, 1.0, 1.0, dn=False), t, wide, 1.0, 1.0, dn=False)


def test_gradient_formula_against_differences():
    rng = np.random.default_rng(0)
    T, d = 3, 7
    for gate in ("row", "all"):
        a = inputs(T, d, "fp32", gate, True, True)
        names = ["y", "res", "gate", "w_post", "w_pre"]
        # everything in float64, h not rounded
        v = {k: a[k].double() for k in names}
        c, e = torch.from_numpy(rng.standard_normal((T, d))), torch.from_numpy(rng.standard_normal((T, d)))

        def loss(q):
            h = forward(q, 0.9, 0.7)["h"]
            n = forward(q, 0.9, 0.7, h=torch.from_numpy(h))["n"]
            return (h * c.numpy()).sum() + (n * e.numpy()).sum()

        b, _ = backward(dict(v, dh=c, dn=e), torch.from_numpy(forward(v, 0.9, 0.7)["h"]), 0.9, 0.7)
        for k, g in (("y", b["dy"]), ("res", b["dres"]), ("w_post", b["dw_post"]), ("w_pre", b["dw_pre"]),
                     ("gate", b["dgate"] if gate == "row" else b["dgate_all"])):
            ref = np.empty(v[k].numel())
            for i in range(v[k].numel()):
                q = {n: x.clone() for n, x in v.items()}
                q[k].view(-1)[i] += 1e-6
                up = loss(q)
                q[k].view(-1)[i] -= 2e-6
                ref[i] = (up - loss(q)) / 2e-6
            assert np.abs(ref.reshape(g.shape) - g).max() < 1e-7, k


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 2048, 7168, 100])
def test_rows_at_the_ends_of_the_range(d, dtype):
    """Rows of zeros, of 1e-40 (eps 0: 1 / rms is past float32) and of 1e38; others are not touched."""
    import routing_grouped_expert_gemm_amd as mok
    t = TYPES[dtype]
    T, wide = 6, 2
    a = inputs(T, d, dtype, "all", True, True, seed=3)
    a["y"][1], a["res"][1] = 0, 0
    a["y"][2] = (a["y"][2].float() * 1e-39).to(t)
    a["y"][3] = (a["y"][3].float().clamp(-1.5, 1.5) * 1e38).to(t)
    a["y"][4], a["res"][4] = (a["y"][4].float() * 1e-39).to(t), (a["res"][4].float() * 1e-39).to(t)
    for k in ("dh", "dn"):
        a[k][4] = 0
    D = {k: None if v is None else v.to(DEV) for k, v in a.items()}
    o = call(mok, D, T, d, t, 1.0, 1.0)                # eps > 0: rows of nothing norm to zero
    for k in o:
        assert torch.isfinite(o[k]).all(), k
    assert (o["n"][1] == 0).all() and (o["h"][1] == 0).all()
    rows = [0, 2, 3, 5]
    sub = {k: v[rows] if v is not None and v.dim() == 2 else v for k, v in a.items()}
    keep = {k: v[rows].to(DEV) if v is not None and v.dim() == 2 else None if v is None else v.to(DEV) for k, v in a.items()}
    o = call(mok, keep, 4, d, t, 1.0, 1.0, eps=0.0)
    assert torch.isinf(o["rstd_y"][1]) and torch.isfinite(o["dw_post"]).all()
    f = forward(sub, 1.0, 1.0, 0.0, o["h"])
    near(o["h"], f["h"], 8 * U * f["h_scale"], t)
    near(o["n"], f["n"], 4 * U * np.abs(f["n"]), t)
    b, s = backward(sub, o["h"], 1.0, 1.0, eps=0.0)
    # a gradient of 1e39 and more leaves the type: only the rows whose own stays inside
    for r in (0, 2, 3):
        near(o["dy"][r:r + 1], b["dy"][r:r + 1], wide * 512 * U * s["dy"][r:r + 1], t)
    near(o["dres"], b["dres"], wide * 136 * U * s["dres"], t)
    near(o["dw_post"], b["dw_post"], wide * 256 * U * s["dw_post"], torch.float32)
    near(o["dgate"], b["dgate_all"], wide * 256 * U * s["dgate_all"], torch.float32)


def test_in_place_and_any_address():
    """h over y or residual, n over the other; tensors 2 bytes off give the aligned ones' result."""
    import routing_grouped_expert_gemm_amd as mok
    for T, d in ((5, 512), (3, 7168), (4, 100)):
        a = inputs(T, d, "bf16", "row", True, True)
        D = {k: v.to(DEV) for k, v in a.items()}
        h, n = torch.empty_like(D["y"]), torch.empty_like(D["y"])
        kw = dict(w_post=D["w_post"], gate=D["gate"], w_pre=D["w_pre"], alpha=0.5, beta=2.0)
        mok.mok_gated_norm(D["y"], D["res"], EPS, h, n=n, **kw)
        for hy in (True, False):
            y, res = D["y"].clone(), D["res"].clone()
            ho, no = (y, res) if hy else (res, y)
            mok.mok_gated_norm(y, res, EPS, ho, n=no, **kw)
            torch.cuda.synchronize()
            assert torch.equal(ho, h) and torch.equal(no, n)
        off = {}
        for k, v in D.items():
            buf = torch.empty(v.numel() + 1, dtype=v.dtype, device=DEV)
            off[k] = buf[1:].view(v.shape).copy_(v)
        h1 = torch.empty(T * d + 1, dtype=torch.bfloat16, device=DEV)[1:].view(T, d)
        n1 = torch.empty(T * d + 1, dtype=torch.bfloat16, device=DEV)[1:].view(T, d)
        mok.mok_gated_norm(off["y"], off["res"], EPS, h1, n=n1, w_post=off["w_post"], gate=off["gate"], w_pre=off["w_pre"],
                           alpha=0.5, beta=2.0)
        torch.cuda.synchronize()
        assert torch.equal(h1, h) and torch.equal(n1, n)      # the same float64 statistics, up to their last bits


def test_no_rows():
    import routing_grouped_expert_gemm_amd as mok
    d = 64
    e, w = torch.empty(0, d, device=DEV), torch.ones(d, device=DEV)
    r = torch.empty(0, device=DEV)
    mok.mok_gated_norm(e, e, EPS, e, w_post=w, w_pre=w, n=e)
    sums = [torch.full((d,), 5.0, device=DEV) for _ in range(3)]
    ws = torch.empty(mok.mok_gated_norm_backward_workspace_bytes(0, d), dtype=torch.uint8, device=DEV)
    mok.mok_gated_norm_backward(e, e, e, e, ws, dn=e, h=e, gate=w, w_post=w, w_pre=w, rstd_y=r, rstd_h=r, dgate=sums[0],
                                dw_post=sums[1], dw_pre=sums[2])
    torch.cuda.synchronize()
    assert all((s == 0).all() for s in sums)


def test_many_rows():
    """More rows than a launch of one workgroup a row takes; the last rows and the sums' counts."""
    import routing_grouped_expert_gemm_amd as mok
    T, d = (1 << 21) + 70, 8
    y = torch.ones(T, d, device=DEV)
    res = torch.zeros(T, d, device=DEV)
    w = torch.full((d,), 2.0, device=DEV)
    h, n, rs = torch.empty_like(y), torch.empty_like(y), [torch.empty(T, device=DEV) for _ in range(2)]
    mok.mok_gated_norm(y, res, 0.0, h, w_post=w, w_pre=w, n=n, rstd_y=rs[0], rstd_h=rs[1])
    dw = [torch.empty(d, device=DEV) for _ in range(2)]
    dy, dres = torch.full_like(y, 9.0), torch.full_like(y, 9.0)
    ws = torch.empty(mok.mok_gated_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_gated_norm_backward(y, y, dres, dy, ws, dn=y, h=h, w_post=w, w_pre=w, rstd_y=rs[0], rstd_h=rs[1], dw_post=dw[0],
                                dw_pre=dw[1])
    torch.cuda.synchronize()
    assert (h == 2).all() and (n == 2).all() and (dres == 1).all() and (dy == 0).all()
    assert (dw[0] == T).all() and (dw[1] == T).all()


def test_captured_and_replayed():
    import routing_grouped_expert_gemm_amd as mok
    T, d = 600, 1536
    a = inputs(T, d, "bf16", "all", True, True)
    D = {k: v.to(DEV) for k, v in a.items()}
    f = dict(device=DEV)
    ws = torch.empty(mok.mok_gated_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)

    def outs():
        return dict(h=torch.empty_like(D["y"]), n=torch.empty_like(D["y"]), ry=torch.empty(T, **f), rh=torch.empty(T, **f),
                    dres=torch.empty_like(D["y"]), dy=torch.empty_like(D["y"]), dg=torch.empty(d, **f),
                    dwa=torch.empty(d, **f), dwb=torch.empty(d, **f))

    def go(o):
        mok.mok_gated_norm(D["y"], D["res"], EPS, o["h"], w_post=D["w_post"], gate=D["gate"], w_pre=D["w_pre"], n=o["n"],
                           rstd_y=o["ry"], rstd_h=o["rh"])
        mok.mok_gated_norm_backward(D["dh"], D["y"], o["dres"], o["dy"], ws, dn=D["dn"], h=o["h"], gate=D["gate"],
                                    w_post=D["w_post"], w_pre=D["w_pre"], rstd_y=o["ry"], rstd_h=o["rh"], dgate=o["dg"],
                                    dw_post=o["dwa"], dw_pre=o["dwb"])

    o, e = outs(), outs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(o)
    for i in range(4):
        for k in ("y", "res", "dh", "dn"):
            D[k].normal_()
        graph.replay()
        torch.cuda.synchronize()
        go(e)
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], e[k]) for k in o), i
