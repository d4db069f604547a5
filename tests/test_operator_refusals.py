"""What the operators around the layer refuse, checked without a GPU: the C entry points return
their status before any launch (pointers here are never followed), and the Python entry points
refuse tensors they cannot marshal."""
import ctypes

import pytest
import torch

P, I64, I32, SZ, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                      ctypes.c_float)
OK, EINVAL, EUNSUPPORTED, EWORKSPACE = 0, 1, 2, 3
BIG = 1 << 40


@pytest.fixture(scope="module")
def mok():
    import routing_grouped_expert_gemm_amd as m
    return m


@pytest.fixture(scope="module")
def lib(mok):
    L = ctypes.CDLL(mok.LIB_PATH)
    L.mok_balance_loss.argtypes = [P, P, I64, I32, I32, P, I32, F, P, P, P, P, SZ, P]
    L.mok_balance_loss_backward.argtypes = [P, P, I64, I32, I32, P, I32, F, P, P, P]
    L.mok_rmsnorm.argtypes = [P, P, P, I64, I32, I32, F, P, P, P, P, P, P]
    L.mok_rmsnorm_backward.argtypes = [P, P, P, P, P, I64, I32, I32, P, P, P, SZ, P]
    L.mok_route_backward.argtypes = [P] * 7 + [I64] + [I32] * 4 + [P, P, P, SZ, P]
    L.mok_mx_gemm.argtypes = [P, P, I32, P, P, I32, I64, I64, I32, I32, P, P, SZ, P]
    return L


def refuse(f, base, status, **kw):
    args = dict(base)
    assert set(kw) <= set(args)
    args.update(kw)
    assert f(*args.values(), None) == status, kw


def test_balance_loss(lib):
    b = dict(logits=16, idx=16, T=10, E=8, k=2, off=16, S=3, alpha=0.1, loss=16, counts=16,
             mean=16, ws=16, ws_bytes=BIG)
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(S=0),
               dict(S=65536), dict(off=None), dict(logits=None), dict(idx=None), dict(loss=None),
               dict(counts=None), dict(mean=None), dict(E=1024, k=65), dict(T=1 << 30)):
        refuse(lib.mok_balance_loss, b, EINVAL, **kw)
    for kw in (dict(ws=None), dict(ws_bytes=100), dict(ws=20)):
        refuse(lib.mok_balance_loss, b, EWORKSPACE, **kw)


def test_balance_loss_backward(lib):
    b = dict(logits=16, counts=16, T=10, E=8, k=2, off=16, S=3, alpha=0.1, dloss=16, dlogits=16)
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(S=0),
               dict(off=None), dict(logits=None), dict(counts=None), dict(dloss=None),
               dict(dlogits=None)):
        refuse(lib.mok_balance_loss_backward, b, EINVAL, **kw)
    refuse(lib.mok_balance_loss_backward, b, OK, T=0, logits=None)


def test_rmsnorm(lib):
    b = dict(x=16, res=None, w=16, rows=4, d=64, io=1, eps=1e-6, h=None, rstd=None, y=16,
             codes=16, scales=16)
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=(1 << 24) + 1), dict(io=2),
               dict(eps=-1.0), dict(eps=float("nan")), dict(codes=None), dict(scales=None),
               dict(d=40), dict(x=None), dict(w=None),
               dict(y=None, codes=None, scales=None)):
        refuse(lib.mok_rmsnorm, b, EINVAL, **kw)
    refuse(lib.mok_rmsnorm, b, OK, rows=0, x=None)


def test_rmsnorm_backward(lib):
    b = dict(dy=16, h=16, rstd=16, w=16, dh=None, rows=4, d=64, io=0, dx=16, dw=16, ws=16,
             ws_bytes=BIG)
    for kw in (dict(rows=-1), dict(d=0), dict(io=3), dict(dy=None), dict(h=None),
               dict(rstd=None), dict(w=None), dict(dx=None)):
        refuse(lib.mok_rmsnorm_backward, b, EINVAL, **kw)
    for kw in (dict(ws=None), dict(ws_bytes=64), dict(ws=24)):
        refuse(lib.mok_rmsnorm_backward, b, EWORKSPACE, **kw)
    refuse(lib.mok_rmsnorm_backward, b, OK, rows=0, dw=None)


def test_route_backward(lib):
    b = dict(x=16, w=16, idx=16, tw=16, dtw=16, dl=None, dx_in=None, T=10, d=64, E=8, k=2, io=1,
             dx=16, dw=16, ws=16, ws_bytes=BIG)
    for kw in (dict(T=-1), dict(d=0), dict(d=(1 << 24) + 1), dict(E=0), dict(E=1025), dict(k=0),
               dict(k=9), dict(E=1024, k=65), dict(io=2), dict(dx=None, dw=None), dict(x=None),
               dict(w=None), dict(idx=None), dict(tw=None), dict(dtw=None), dict(T=1 << 30)):
        refuse(lib.mok_route_backward, b, EINVAL, **kw)
    for kw in (dict(ws=None), dict(ws_bytes=8), dict(ws=24)):
        refuse(lib.mok_route_backward, b, EWORKSPACE, **kw)
    refuse(lib.mok_route_backward, b, EUNSUPPORTED, T=1 << 29, d=1 << 16, k=1, w=16)


def test_mx_gemm(lib):
    b = dict(a=16, asc=16, fa=3, b=16, bsc=16, fb=3, M=100, N=64, K=4096, out=1, c=16, ws=16,
             ws_bytes=BIG)
    for kw in (dict(M=-1), dict(N=-1), dict(M=1 << 31), dict(N=1 << 31), dict(K=0), dict(K=33),
               dict(K=(1 << 22) + 32), dict(fa=1), dict(fb=0), dict(out=2), dict(a=None),
               dict(asc=None), dict(b=None), dict(bsc=None), dict(c=None), dict(a=24),
               dict(b=17), dict(c=18)):
        refuse(lib.mok_mx_gemm, b, EINVAL, **kw)
    for kw in (dict(ws=None), dict(ws_bytes=64), dict(ws=24)):
        refuse(lib.mok_mx_gemm, b, EWORKSPACE, **kw)
    refuse(lib.mok_mx_gemm, b, EUNSUPPORTED, M=(1 << 31) - 1, N=(1 << 31) - 1)
    refuse(lib.mok_mx_gemm, b, EUNSUPPORTED, M=1, N=1 << 28)
    refuse(lib.mok_mx_gemm, b, OK, M=0, a=None, c=None)


def test_workspace_queries(mok):
    assert mok.mok_balance_loss_workspace_bytes(0, 8, 1) > 0
    assert mok.mok_rmsnorm_backward_workspace_bytes(0, 64) >= 256
    assert mok.mok_route_backward_workspace_bytes(1, 64, 8, torch.bfloat16) > 0
    assert mok.mok_mx_gemm_workspace_bytes(1, 64, 64) == 0
    assert mok.mok_mx_gemm_workspace_bytes(0, 64, 64) == 0
    for f, args in ((mok.mok_balance_loss_workspace_bytes, (-1, 8, 1)),
                    (mok.mok_balance_loss_workspace_bytes, (8, 2000, 1)),
                    (mok.mok_balance_loss_workspace_bytes, (8, 8, 0)),
                    (mok.mok_rmsnorm_backward_workspace_bytes, (-1, 8)),
                    (mok.mok_route_backward_workspace_bytes, (8, 8, 8, torch.float16)),
                    (mok.mok_mx_gemm_workspace_bytes, (8, 8, 40))):
        with pytest.raises(mok.MokError) as e:
            f(*args)
        assert e.value.status == EINVAL


def test_tensors_that_cannot_be_marshalled(mok):
    """Host tensors reach no kernel (a wrong type, shape or stride is refused in the same place,
    before the device is looked at)."""
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    u = torch.zeros(4, 32, dtype=torch.uint8)
    calls = [
        lambda: mok.mok_balance_loss(f, i, 0.1, f[0, :1], i[:1], f[:1], u),
        lambda: mok.mok_balance_loss(f[0], i, 0.1, f[0, :1], i[:1], f[:1], u),
        lambda: mok.mok_balance_loss_backward(f, i, 2, 0.1, f[0, :1], f),
        lambda: mok.mok_rmsnorm(f, f[0], 1e-6, y=f),
        lambda: mok.mok_rmsnorm(f.half(), f[0], 1e-6, y=f),
        lambda: mok.mok_rmsnorm_backward(f, f, f[:, 0], f[0], f),
        lambda: mok.mok_route_backward(f, f, i, f[:, :2], f[:, :2], f, f, u),
        lambda: mok.mok_mx_gemm(u, u[:, :2], u, u[:, :2], f, u),
        lambda: mok.mok_mx_gemm(u, u[:, :3], u, u[:, :2], f, u),
    ]
    for c in calls:
        with pytest.raises(mok.MokError) as e:
            c()
        assert e.value.status == EINVAL
