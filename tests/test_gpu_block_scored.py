"""The operators of the block together, as they are used.

Training: gated norm (the block before) -> router with scores, bias and groups -> balance loss ->
experts -> gated norm of the layer's output -> next norm; then the way back. Against float64 autograd of
the same formulas with the picks held fixed, on the values that the forward stored in bf16. Serving:
norm -> router -> experts on 4-bit weights over a shared expert on 4-bit products -> gated norm.

Tolerances. Every tensor that passes between two steps is bf16 (half a step is 2^-8 of a value; over
many values of random signs about 2^-8 / sqrt(3) of the tensor's norm). A gradient passes at most 10 of
them on its way (dy of the last norm, dP, G and U's product H, dG and dU, the slots' dx, their sum, dx,
the first norm's dres and dy, the stored n), each of them off by the product of two or three such
roundings at most: 10 * 3 * 2^-8 / sqrt(3) < 0.07 of the reference's norm. Serving: 6 tensors: < 0.041."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def off(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


def rms(v, w, eps):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + eps) * w


def ffn(a, g, u, d):
    return (torch.nn.functional.silu(a @ g.T) * (a @ u.T)) @ d.T


def test_training_step():
    import routing_grouped_expert_gemm_amd as mok
    T, d, E, k, I, alpha, eps = 384, 256, 16, 4, 128, 0.5, 1e-6
    rule = dict(score="sigmoid", renorm=True, scale=2.5)
    groups = dict(n_groups=4, topk_groups=2, group_top=2)
    g = torch.Generator().manual_seed(21)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).bfloat16()  # noqa: E731
    one = lambda: (1 + 0.1 * torch.randn(d, generator=g)).bfloat16()  # noqa: E731
    a0, res, gate = rnd(T, d), rnd(T, d), torch.sigmoid(torch.randn(T, d, generator=g)).bfloat16()
    w1, w2, w3, w4, gate2 = one(), one(), one(), one(), one()
    wr, bias = rnd(E, d, scale=d ** -0.5), 0.05 * torch.randn(E, generator=g)
    wg, wu, wd = rnd(E, I, d, scale=d ** -0.5), rnd(E, I, d, scale=d ** -0.5), rnd(E, d, I, scale=I ** -0.5)
    dh2, dn2 = rnd(T, d), rnd(T, d)
    D = lambda t: t.to(DEV)  # noqa: E731
    bf, f32, i32 = dict(dtype=torch.bfloat16, device=DEV), dict(device=DEV), dict(dtype=torch.int32, device=DEV)
    rows = lambda: torch.empty(T, d, **bf)  # noqa: E731
    u8 = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)  # noqa: E731

    # forward: join the block before, route its norm, experts, join their output
    h1, n1, ry1, rh1 = rows(), rows(), torch.empty(T, **f32), torch.empty(T, **f32)
    j1 = dict(gate=D(gate), w_post=D(w1), w_pre=D(w2), alpha=1.0, beta=0.7)
    mok.mok_gated_norm(D(a0), D(res), eps, h1, n=n1, rstd_y=ry1, rstd_h=rh1, **j1)
    logits, idx, tw = torch.empty(T, E, **f32), torch.empty(T, k, **i32), torch.empty(T, k, **f32)
    mok.mok_route_scored(n1, D(wr), k, logits, idx, tw, bias=D(bias), **rule, **groups)
    loss, counts, mean = torch.empty(1, **f32), torch.empty(1, E, **i32), torch.empty(1, E, **f32)
    mok.mok_balance_loss(logits, idx, alpha, loss, counts, mean, u8(mok.mok_balance_loss_workspace_bytes(T, E, 1)))
    common = dict(d=d, E=E, k=k, I=I, e0=0, E_l=E, tokens_per_rank=T, T_pool=T, own_begin=0, T_own=T, n_shared=0,
                  I_shared=0, x=n1, topk_idx=idx, topk_w=tw, w_gate=D(wg), w_up=D(wu), w_down=D(wd))
    layer = mok.MoeLayer(dtype="bf16", minibatch_rows=128, ring_rows=1024, **common)
    layer.forward()
    h2, n2, ry2, rh2 = rows(), rows(), torch.empty(T, **f32), torch.empty(T, **f32)
    j2 = dict(gate=D(gate2), w_post=D(w3), w_pre=D(w4), alpha=0.9, beta=1.0)
    mok.mok_gated_norm(layer.y, h1, eps, h2, n=n2, rstd_y=ry2, rstd_h=rh2, **j2)
    # backward
    ws = u8(mok.mok_gated_norm_backward_workspace_bytes(T, d))
    dh1, dy, dg2, dw3, dw4 = rows(), rows(), torch.empty(d, **f32), torch.empty(d, **f32), torch.empty(d, **f32)
    mok.mok_gated_norm_backward(D(dh2), layer.y, dh1, dy, ws, dn=D(dn2), h=h2, rstd_y=ry2, rstd_h=rh2, dgate=dg2,
                                dw_post=dw3, dw_pre=dw4, **j2)
    bwd = mok.MoeBackward(dy=dy, **common)
    bwd.backward()
    dl = torch.empty(T, E, **f32)
    mok.mok_balance_loss_backward(logits, counts, k, alpha, torch.ones(1, **f32), dl)
    mok.mok_topk_scored_backward(logits, idx, bwd.dtopk_w, dl, dlogits_in=dl, **rule)
    dwr = torch.empty(E, d, **f32)
    mok.mok_route_backward(n1, D(wr), None, None, None, bwd.dx, dwr,
                           u8(mok.mok_route_backward_workspace_bytes(T, d, E, n1.dtype)), dlogits=dl, dx_in=bwd.dx)
    dres, da0, dg1, dw1, dw2 = rows(), rows(), rows(), torch.empty(d, **f32), torch.empty(d, **f32)
    mok.mok_gated_norm_backward(dh1, D(a0), dres, da0, ws, dn=bwd.dx, h=h1, rstd_y=ry1, rstd_h=rh1, dgate=dg1,
                                dw_post=dw1, dw_pre=dw2, **j1)
    torch.cuda.synchronize()
    assert layer.device_error() == 0 and bwd.device_error() == 0

    # the picks are those of the definition, on the logits that the router gave
    lg = logits.cpu().double()
    c = torch.sigmoid(lg) + bias.double()
    worth = c.view(T, 4, 4).topk(2, dim=2).values.sum(2)
    keep = torch.zeros(T, 4).scatter_(1, worth.topk(2, dim=1).indices, 1.0).bool().repeat_interleave(4, 1)
    assert torch.equal(idx.cpu().long(), c.masked_fill(~keep, -1e9).topk(k, dim=1).indices)

    # float64 autograd, picks fixed
    L = {n: t.double().requires_grad_() for n, t in
         dict(a0=a0, res=res, gate=gate, w1=w1, w2=w2, w3=w3, w4=w4, g2=gate2, wr=wr, wg=wg, wu=wu, wd=wd).items()}
    ix = idx.cpu().long()
    H1 = L["res"] + 0.7 * L["gate"] * rms(L["a0"], L["w1"], eps)
    N1 = rms(H1, L["w2"], eps)
    lr = N1 @ L["wr"].T
    p = torch.gather(torch.sigmoid(lr), 1, ix)
    w = 2.5 * p / p.sum(1, keepdim=True)
    y = 0
    for e in range(E):
        y = y + torch.where(ix == e, w, 0.0).sum(1, keepdim=True) * ffn(N1, L["wg"][e], L["wu"][e], L["wd"][e])
    H2 = 0.9 * H1 + L["g2"] * rms(y, L["w3"], eps)
    N2 = rms(H2, L["w4"], eps)
    cnt = torch.bincount(ix.reshape(-1), minlength=E).double()
    bal = alpha * (cnt * E / (k * T) * torch.softmax(lr, 1).mean(0)).sum()
    ((H2 * dh2.double()).sum() + (N2 * dn2.double()).sum() + bal).backward()
    assert torch.equal(counts[0].cpu().double(), cnt)
    for got, ref in ((h1, H1), (n1, N1), (h2, H2), (n2, N2), (tw, w)):
        assert off(got, ref.detach()) <= 0.02
    for got, name in ((da0, "a0"), (dres, "res"), (dg1, "gate"), (dw1, "w1"), (dw2, "w2"), (dw3, "w3"), (dw4, "w4"),
                      (dg2, "g2"), (dwr, "wr"), (bwd.dw_gate, "wg"), (bwd.dw_up, "wu"), (bwd.dw_down, "wd")):
        assert off(got, L[name].grad) <= 0.07, name


@pytest.mark.parametrize("T", [1, 5, 40])
def test_serving_step(T):
    import routing_grouped_expert_gemm_amd as mok
    d, E, k, I, I_sh, group, eps = 512, 32, 4, 256, 384, 128, 1e-6
    g = torch.Generator().manual_seed(T)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).bfloat16()  # noqa: E731
    x, res, w1, w2, w3 = rnd(T, d), rnd(T, d), 1 + 0.1 * rnd(d), 1 + 0.1 * rnd(d), 1 + 0.1 * rnd(d)
    wr, bias, gate = rnd(E, d, scale=d ** -0.5), 0.05 * torch.randn(E, generator=g), torch.sigmoid(rnd(T, d).float()).bfloat16()
    raw = dict(gate=rnd(E * I, d, scale=d ** -0.5), up=rnd(E * I, d, scale=d ** -0.5), down=rnd(E * d, I, scale=I ** -0.5),
               sg=rnd(I_sh, d, scale=d ** -0.5), su=rnd(I_sh, d, scale=d ** -0.5), sd=rnd(d, I_sh, scale=I_sh ** -0.5))
    D = lambda t: t.to(DEV)  # noqa: E731
    bf, f32 = dict(dtype=torch.bfloat16, device=DEV), dict(device=DEV)
    q, value = {}, {}
    for n, w in raw.items():                              # weights quantised once
        N, K = w.shape
        c, s = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV), torch.empty(N, K // group, **bf)
        z = torch.empty(N, K // group, dtype=torch.uint8, device=DEV)
        mok.mok_quantize_int4(D(w), c, s, z)
        q[n] = (c, s, z)
        v = torch.stack([c & 15, c >> 4], -1).flatten(-2).cpu().double()
        value[n] = (v - z.cpu().double().repeat_interleave(group, 1)) * s.cpu().double().repeat_interleave(group, 1)
        assert off(value[n], w.double()) < 0.12
    lead = lambda n, a: tuple(t.view(E, a, -1) for t in q[n])  # noqa: E731
    layer = mok.MoeW4Layer(lead("gate", I), lead("up", I), lead("down", d), E=E, k=k, max_tokens=T)
    h, n1, logits = torch.empty(T, d, **bf), torch.empty(T, d, **bf), torch.empty(T, E, **f32)
    idx, tw = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, **f32)
    mok.mok_rmsnorm(D(x), D(w1), eps, residual=D(res), h=h, y=n1)
    mok.mok_route_scored(n1, D(wr), k, logits, idx, tw, bias=D(bias), n_groups=8, topk_groups=4, scale=2.5)
    sh = [torch.empty(T, I_sh, **f32) for _ in range(2)]
    for n, o in zip(("sg", "su"), sh):
        mok.mok_w4_gemm(n1, *q[n][:2], o, zeros=q[n][2])
    a = (torch.nn.functional.silu(sh[0]) * sh[1]).bfloat16()
    y = torch.empty(T, d, **bf)
    mok.mok_w4_gemm(a, *q["sd"][:2], y, zeros=q["sd"][2])
    layer.forward(n1, idx, tw, y, y_in=y)
    h2, n2 = torch.empty(T, d, **bf), torch.empty(T, d, **bf)
    mok.mok_gated_norm(y, h, eps, h2, w_post=D(w2), gate=D(gate), w_pre=D(w3), n=n2)
    torch.cuda.synchronize()
    H = (x.double() + res.double()).bfloat16().double()
    N1 = rms(H, w1.double(), eps)
    ref = ffn(N1, value["sg"], value["su"], value["sd"])
    ix, p = idx.cpu().long(), torch.gather(torch.sigmoid(N1 @ wr.double().T), 1, idx.cpu().long())
    w = 2.5 * p / p.sum(1, keepdim=True)
    W = {n: value[n].view(E, -1, value[n].shape[1]) for n in ("gate", "up", "down")}
    for t in range(T):
        for j in range(k):
            e = ix[t, j]
            ref[t] += w[t, j] * ffn(N1[t:t + 1], W["gate"][e], W["up"][e], W["down"][e])[0]
    H2 = H + gate.double() * rms(ref, w2.double(), eps)
    for got, r in ((tw, w), (y, ref), (h2, H2), (n2, rms(H2, w3.double(), eps))):
        assert off(got, r) <= 0.041
