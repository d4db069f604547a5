"""The operators around the layer together with the layer itself, as one training step of a block
uses them: residual norm -> router -> balance loss -> experts, then the way back: experts' backward,
balance loss's, router's, norm's. Against float64 autograd of the same formulas with the picks held
fixed, on the values that the forward stored in bf16; and the serving form: norm with MXFP8 output
into the product with an MXFP4 weight.

Tolerances. Every tensor that passes between two steps is bf16 (half a step is 2^-8 of a value; in
the norm of a difference over many values of random signs about 2^-8 / sqrt(3) of the tensor's
norm), and a gradient passes through at most 8 of them on its way (dy, dP, G and U's product H, dG and dU,
the slots' dx, their sum, dx, the norm's dx), each of them off by the product of two or three such
roundings at most: 8 * 3 * 2^-8 / sqrt(3) < 0.055 of the reference's norm. Float32 results that see
no such chain (loss, counts, mean probabilities) keep the bounds of their own tests."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def off(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


def test_training_step():
    import routing_grouped_expert_gemm_amd as mok
    T, d, E, k, I, n_sh, I_sh, alpha, eps = 384, 256, 8, 2, 128, 1, 128, 0.5, 1e-6
    g = torch.Generator().manual_seed(11)

    def rnd(*s, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*s, generator=g) * scale).to(dtype)

    x, res, wn = rnd(T, d), rnd(T, d), (1 + 0.1 * torch.randn(d, generator=g)).bfloat16()
    wr = rnd(E, d, scale=d ** -0.5)
    wg, wu, wd = rnd(E, I, d, scale=d ** -0.5), rnd(E, I, d, scale=d ** -0.5), rnd(E, d, I, scale=I ** -0.5)
    sg, su, sd = (rnd(n_sh, I_sh, d, scale=d ** -0.5), rnd(n_sh, I_sh, d, scale=d ** -0.5),
                  rnd(n_sh, d, I_sh, scale=I_sh ** -0.5))
    dy, dh = rnd(T, d), rnd(T, d)
    off_seq = [0, 100, 100, 350]
    D = lambda t: t.to(DEV)  # noqa: E731
    f32, i32 = dict(device=DEV), dict(dtype=torch.int32, device=DEV)
    S = len(off_seq) - 1
    so = torch.tensor(off_seq, **i32)

    # forward
    h, y = torch.empty(T, d, dtype=torch.bfloat16, device=DEV), torch.empty(
        T, d, dtype=torch.bfloat16, device=DEV)
    rstd = torch.empty(T, **f32)
    mok.mok_rmsnorm(D(x), D(wn), eps, residual=D(res), h=h, y=y, rstd=rstd)
    layer = mok.MoeLayer(dtype="bf16", d=d, E=E, k=k, I=I, e0=0, E_l=E, tokens_per_rank=T, T_pool=T,
                         own_begin=0, T_own=T, n_shared=n_sh, I_shared=I_sh, minibatch_rows=128,
                         ring_rows=1024, x=y, w_router=D(wr), w_gate=D(wg), w_up=D(wu), w_down=D(wd),
                         ws_gate=D(sg), ws_up=D(su), ws_down=D(sd), keep_intermediates=True, device=DEV)
    layer.forward()
    logits, idx, tw = (layer.inter[n] for n in ("logits", "topk_idx", "topk_w"))
    loss, counts, mean = torch.empty(1, **f32), torch.empty(S, E, **i32), torch.empty(S, E, **f32)
    ws = torch.empty(mok.mok_balance_loss_workspace_bytes(T, E, S), dtype=torch.uint8, device=DEV)
    mok.mok_balance_loss(logits, idx, alpha, loss, counts, mean, ws, seq_offsets=so)
    # backward
    bwd = mok.MoeBackward(d=d, E=E, k=k, I=I, e0=0, E_l=E, tokens_per_rank=T, T_pool=T, own_begin=0,
                          T_own=T, n_shared=n_sh, I_shared=I_sh, x=y, topk_idx=idx, topk_w=tw,
                          w_gate=D(wg), w_up=D(wu), w_down=D(wd), ws_gate=D(sg), ws_up=D(su),
                          ws_down=D(sd), dy=D(dy))
    bwd.backward()
    dlogits, dwr = torch.empty(T, E, **f32), torch.empty(E, d, **f32)
    mok.mok_balance_loss_backward(logits, counts, k, alpha, torch.ones(1, **f32), dlogits,
                                  seq_offsets=so)
    ws2 = torch.empty(mok.mok_route_backward_workspace_bytes(T, d, E, y.dtype), dtype=torch.uint8,
                      device=DEV)
    mok.mok_route_backward(y, D(wr), idx, tw, bwd.dtopk_w, bwd.dx, dwr, ws2, dlogits=dlogits,
                           dx_in=bwd.dx)
    dx, dwn = torch.empty_like(h), torch.empty(d, **f32)
    ws3 = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_rmsnorm_backward(bwd.dx, h, rstd, D(wn), dx, dwn, ws3, dh=D(dh))
    torch.cuda.synchronize()
    assert layer.device_error() == 0 and bwd.device_error() == 0

    # float64 autograd, picks fixed
    L = {n: t.double().requires_grad_() for n, t in
         dict(h=h.cpu(), wn=wn, wr=wr, wg=wg, wu=wu, wd=wd, sg=sg, su=su, sd=sd).items()}
    ix = idx.cpu().long()
    yr = L["h"] * torch.rsqrt((L["h"] ** 2).mean(1, keepdim=True) + eps) * L["wn"]
    lg = yr @ L["wr"].T
    w = torch.softmax(torch.gather(lg, 1, ix), 1)
    ffn = lambda a, gw, uw, dw: (torch.nn.functional.silu(a @ gw.T) * (a @ uw.T)) @ dw.T  # noqa: E731
    out = ffn(yr, L["sg"][0], L["su"][0], L["sd"][0])
    for e in range(E):
        we = torch.where(ix == e, w, 0.0).sum(1, keepdim=True)
        out = out + we * ffn(yr, L["wg"][e], L["wu"][e], L["wd"][e])
    bal = 0.0
    for s in range(S):
        a, b = off_seq[s], off_seq[s + 1]
        if b > a:
            c = torch.bincount(ix[a:b].reshape(-1), minlength=E).double()
            assert torch.equal(counts[s].cpu().double(), c)
            bal = bal + alpha / S * (c * E / (k * (b - a)) * torch.softmax(lg[a:b], 1).mean(0)).sum()
    ((out * dy.double()).sum() + bal + (L["h"] * dh.double()).sum()).backward()
    bal = float(bal.detach())
    assert abs(float(loss) - bal) <= 2.0 ** -8 * abs(bal)       # logits of bf16 rows
    assert off(y, yr.detach()) <= 2.0 ** -8
    for got, name in ((dx, "h"), (dwn, "wn"), (dwr, "wr"), (bwd.dw_gate, "wg"), (bwd.dws_down, "sd")):
        assert off(got, L[name].grad) <= 0.055, name


@pytest.mark.parametrize("T", [1, 5, 300])
def test_norm_into_product(T):
    """Norm -> MXFP8 rows -> product with an MXFP4 weight: exactly the product of the codes."""
    import oracle
    import routing_grouped_expert_gemm_amd as mok
    d, N = 512, 384
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, d, generator=g).bfloat16().to(DEV), torch.ones(d).bfloat16().to(DEV)
    B = torch.randn(N, d, generator=g).bfloat16().to(DEV)
    u8 = dict(dtype=torch.uint8, device=DEV)
    a, asc = torch.empty(T, d, **u8), torch.empty(T, d // 32, **u8)
    b, bsc = torch.empty(N, d // 2, **u8), torch.empty(N, d // 32, **u8)
    c = torch.empty(T, N, device=DEV)
    mok.mok_quantize_mxfp4(B, b, bsc)
    mok.mok_rmsnorm(x, w, 1e-6, codes=a, scales=asc)
    ws = torch.empty(mok.mok_mx_gemm_workspace_bytes(T, N, d), **u8)
    mok.mok_mx_gemm(a, asc, b, bsc, c, ws)
    torch.cuda.synchronize()
    av = oracle.mxfp8_dequantize(a.cpu().numpy(), asc.cpu().numpy()).astype(np.float64)
    bv = oracle.mxfp4_dequantize(b.cpu().numpy(), bsc.cpu().numpy()).astype(np.float64)
    bound = d * 2.0 ** -23 * (np.abs(av) @ np.abs(bv).T)
    assert (np.abs(c.cpu().double().numpy() - av @ bv.T) <= bound).all()
