"""The routing weights' gradient of shares of the experts, into the router: a share's dtopk_w is zero at
other experts' routes, also when the picks change between calls, and the shares' gradients add up to the
whole layer's."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
U = 2.0 ** -24
T, D, E, K, I = 300, 128, 16, 4, 64


def layer(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, f=1.0: (torch.randn(s, generator=g, device=DEV) * f).to(BF)  # noqa: E731
    top = torch.topk(torch.randn(T, E, generator=g, device=DEV), K, dim=1)
    return dict(x=r(T, D), wr=r(E, D, f=D ** -0.5), wg=r(E, I, D, f=D ** -0.5), wu=r(E, I, D, f=D ** -0.5),
                wd=r(E, D, I, f=I ** -0.5), dy=r(T, D), idx=top.indices.int().contiguous(),
                tw=torch.softmax(top.values, 1).contiguous())


def experts(mok, v, e0, e1):
    whole = e1 - e0 == E
    up = dict(dy=v["dy"]) if whole else dict(
        dy_slots=v["dy"].repeat_interleave(K, 0).contiguous(), dy_shared=v["dy"])
    b = mok.MoeBackward(d=D, E=E, k=K, I=I, e0=e0, E_l=e1 - e0, tokens_per_rank=T, T_pool=T, own_begin=0,
                        T_own=T, n_shared=0, I_shared=0, x=v["x"], topk_idx=v["idx"], topk_w=v["tw"],
                        w_gate=v["wg"][e0:e1].contiguous(), w_up=v["wu"][e0:e1].contiguous(),
                        w_down=v["wd"][e0:e1].contiguous(), device=DEV, **up)
    b.dtopk_w.fill_(float("nan"))                    # what fresh memory may hold
    return b


def into_router(mok, v, dtopk_w):
    dx, dw = torch.empty_like(v["x"]), torch.empty(E, D, device=DEV)
    ws = torch.empty(mok.mok_route_backward_workspace_bytes(T, D, E, BF), dtype=torch.uint8, device=DEV)
    mok.mok_route_backward(v["x"], v["wr"], v["idx"], v["tw"], dtopk_w, dx, dw, ws)
    return dx, dw


@pytest.mark.parametrize("how", ["current", "stream", "handle", "default"])
def test_shares_add_up(how):
    import routing_grouped_expert_gemm_amd as mok
    side = torch.cuda.Stream()
    stream = dict(current=None, stream=side, handle=side.cuda_stream, default=0)[how]
    v = layer(1)
    parts = [(0, 5), (5, 6), (6, 16)]
    shares = [experts(mok, v, *p) for p in parts]
    whole = experts(mok, v, 0, E)
    for seed in (1, 2):                              # the second time with other picks in place
        n = layer(seed)
        v["idx"].copy_(n["idx"])
        v["tw"].copy_(n["tw"])
        torch.cuda.synchronize()
        for b in shares:
            b.backward(stream)
        whole.backward()
        torch.cuda.synchronize()
        for b, (e0, e1) in zip(shares, parts):
            mine = (v["idx"] >= e0) & (v["idx"] < e1)
            assert (b.dtopk_w[~mine] == 0).all()
            assert torch.equal(b.dtopk_w[mine], whole.dtopk_w[mine])
        got = [into_router(mok, v, b.dtopk_w) for b in shares]
        dx, dw = into_router(mok, v, whole.dtopk_w)
        torch.cuda.synchronize()
        # the router backward's bounds, for the whole and for each share: dl is off by (K + 8) U of its
        # absolute terms; dw adds T products, dx E of 16 bits, rounded to bf16
        tw, da = v["tw"].double(), whole.dtopk_w.double().abs()
        D_ = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_add_(
            1, v["idx"].long(), tw * (da + (tw * da).sum(1, keepdim=True)))
        tol = 2 * (T + K + 10) * U * (D_.T.contiguous() @ v["x"].double().abs())
        assert ((sum(g[1].double() for g in got) - dw.double()).abs() <= tol).all()
        s = D_ @ v["wr"].double().abs()
        tol = 2 * ((E + K + 10) * U + 2.0 ** -16) * s + 2.0 ** -8 * (
            dx.double().abs() + sum(g[0].double().abs() for g in got)) * 1.01
        assert ((sum(g[0].double() for g in got) - dx.double()).abs() <= tol).all()
