"""What the operators of the block refuse (choice by scores, gated norm, 4-bit weights), checked
without a GPU: the C entry points return their status before any launch (pointers here are never
followed), and the Python entry points refuse tensors they cannot marshal."""
import ctypes
import os
import subprocess

import pytest
import torch

P, I64, I32, SZ, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                      ctypes.c_float)
OK, EINVAL, EUNSUPPORTED, EWORKSPACE = 0, 1, 2, 3
BIG = 1 << 40
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mok():
    import routing_grouped_expert_gemm_amd as m
    return m


@pytest.fixture(scope="module")
def lib(mok):
    L = ctypes.CDLL(mok.LIB_PATH)
    rule = [I32, P, I32, I32, I32, I32, F]
    L.mok_topk_scored.argtypes = [P, I64, I32, I32] + rule + [P, P, P]
    L.mok_route_scored.argtypes = [P, P, I64] + [I32] * 4 + rule + [P] * 4
    L.mok_topk_scored_backward.argtypes = [P] * 4 + [I64] + [I32] * 4 + [F, P, P]
    L.mok_gated_norm.argtypes = [P, P, P, I32, P, P, I64, I32, I32, F, F, F] + [P] * 5
    L.mok_gated_norm_backward.argtypes = ([P] * 6 + [I32] + [P] * 3 + [I64, I32, I32, F, F]
                                          + [P] * 6 + [SZ, P])
    L.mok_quantize_int4.argtypes = [P, I64, I32, I32, P, P, P, P]
    L.mok_w4_gemm.argtypes = [P] * 4 + [I64, I64, I32, I32, I32, P, P]
    return L


def refuse(f, base, status, **kw):
    args = dict(base)
    assert set(kw) <= set(args)
    args.update(kw)
    assert f(*args.values(), None) == status, kw


NAN, INF = float("nan"), float("inf")
BAD_RULE = (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(k=65), dict(score=2),
            dict(score=-1), dict(G=0), dict(G=3), dict(G=32), dict(Gk=0), dict(Gk=5), dict(Gk=1, k=5),
            dict(top=0), dict(top=3), dict(scale=NAN), dict(scale=INF), dict(T=1 << 30))


def test_topk_scored(lib):
    b = dict(logits=16, T=10, E=16, k=4, score=1, bias=None, G=4, Gk=2, top=2, renorm=1, scale=1.0,
             idx=16, w=16)
    for kw in BAD_RULE + (dict(logits=None), dict(idx=None), dict(w=None)):
        refuse(lib.mok_topk_scored, b, EINVAL, **kw)
    refuse(lib.mok_topk_scored, b, EINVAL, E=1024, G=1, Gk=1, k=65)
    refuse(lib.mok_topk_scored, b, OK, T=0, logits=None)


def test_route_scored(lib):
    b = dict(x=16, wr=16, T=10, d=64, E=16, k=4, io=1, score=1, bias=None, G=4, Gk=2, top=2,
             renorm=1, scale=1.0, logits=16, idx=16, w=16)
    for kw in BAD_RULE + (dict(d=0), dict(io=2), dict(x=None), dict(wr=None), dict(logits=None),
                          dict(idx=None), dict(w=None)):
        refuse(lib.mok_route_scored, b, EINVAL, **kw)
    refuse(lib.mok_route_scored, b, OK, T=0, x=None)


def test_topk_scored_backward(lib):
    b = dict(logits=16, idx=16, dw=16, din=None, T=10, E=16, k=4, score=0, renorm=0, scale=1.0,
             dl=16)
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(score=2),
               dict(scale=NAN), dict(logits=None), dict(idx=None), dict(dw=None), dict(dl=None),
               dict(T=1 << 30)):
        refuse(lib.mok_topk_scored_backward, b, EINVAL, **kw)
    refuse(lib.mok_topk_scored_backward, b, OK, T=0, logits=None)


def test_gated_norm(lib):
    b = dict(y=16, w_post=16, gate=16, per=1, res=16, w_pre=16, rows=4, d=64, io=1, eps=1e-6,
             alpha=1.0, beta=1.0, h=16, n=16, ry=16, rh=16)
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=(1 << 24) + 1), dict(io=2),
               dict(eps=-1.0), dict(eps=NAN), dict(alpha=INF), dict(beta=NAN), dict(y=None),
               dict(res=None), dict(h=None), dict(w_post=None), dict(w_pre=None),
               dict(w_pre=None, n=None), dict(w_pre=None, rh=None)):
        refuse(lib.mok_gated_norm, b, EINVAL, **kw)
    refuse(lib.mok_gated_norm, b, OK, rows=0, y=None)


def test_gated_norm_backward(lib):
    b = dict(dh=16, dn=16, y=16, h=16, w_post=16, gate=16, per=0, w_pre=16, ry=16, rh=16, rows=4,
             d=64, io=0, alpha=1.0, beta=1.0, dres=16, dy=16, dgate=16, dw_post=16, dw_pre=16,
             ws=16, ws_bytes=BIG)
    for kw in (dict(rows=-1), dict(d=0), dict(io=3), dict(alpha=NAN), dict(dh=None, dn=None),
               dict(y=None), dict(h=None), dict(ry=None), dict(rh=None), dict(gate=None),
               dict(w_post=None), dict(w_pre=None), dict(w_pre=None, dn=None),
               dict(w_pre=None, dw_pre=None),
               dict(dres=None, dy=None, dgate=None, dw_post=None, dw_pre=None)):
        refuse(lib.mok_gated_norm_backward, b, EINVAL, **kw)
    for kw in (dict(ws=None), dict(ws_bytes=64), dict(ws=24)):
        refuse(lib.mok_gated_norm_backward, b, EWORKSPACE, **kw)
    refuse(lib.mok_gated_norm_backward, b, OK, rows=0, dgate=None, dw_post=None, dw_pre=None)


def test_quantize_int4(lib):
    b = dict(src=16, rows=3, K=128, group=64, codes=16, scales=16, zeros=None)
    for kw in (dict(rows=-1), dict(K=0), dict(K=96), dict(group=16), dict(group=256), dict(src=None),
               dict(codes=None), dict(scales=None), dict(src=24), dict(codes=18)):
        refuse(lib.mok_quantize_int4, b, EINVAL, **kw)
    refuse(lib.mok_quantize_int4, b, EUNSUPPORTED, rows=1 << 40)
    refuse(lib.mok_quantize_int4, b, OK, rows=0, src=None)


def test_w4_gemm(lib):
    b = dict(x=16, codes=16, scales=16, zeros=None, M=4, N=32, K=128, group=64, out=1, c=16)
    for kw in (dict(M=-1), dict(N=-1), dict(M=1 << 31), dict(K=0), dict(K=96), dict(K=32), dict(group=48),
               dict(K=(1 << 22) + 64), dict(out=2), dict(x=None), dict(codes=None), dict(scales=None),
               dict(c=None), dict(x=24), dict(codes=24), dict(scales=17), dict(c=17), dict(c=18, out=0)):
        refuse(lib.mok_w4_gemm, b, EINVAL, **kw)
    refuse(lib.mok_w4_gemm, b, EUNSUPPORTED, M=(1 << 20) + 1)
    refuse(lib.mok_w4_gemm, b, EUNSUPPORTED, N=(1 << 26) + 1)
    refuse(lib.mok_w4_gemm, b, OK, M=0, x=None)
    refuse(lib.mok_w4_gemm, b, OK, N=0, c=None)


def moe_args(mok, **kw):
    a = mok.MoeW4Args()
    base = dict(T=4, d=128, I=64, E=16, k=4, e0=4, E_l=8, group=64, x=16, topk_idx=16, topk_w=16,
                gate_codes=16, up_codes=16, down_codes=16, gate_scales=16, up_scales=16,
                down_scales=16, y=16, workspace=16, workspace_bytes=BIG)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


def test_moe_w4(mok):
    lib = ctypes.CDLL(mok.LIB_PATH)
    lib.mok_moe_w4_forward.argtypes = [ctypes.POINTER(mok.MoeW4Args), P]
    call = lambda **kw: lib.mok_moe_w4_forward(ctypes.byref(moe_args(mok, **kw)), None)  # noqa: E731
    for kw in (dict(T=-1), dict(d=0), dict(I=0), dict(d=96), dict(I=96), dict(group=0), dict(group=48),
               dict(E=0), dict(k=0), dict(k=17), dict(E=200, k=65), dict(e0=-1), dict(E_l=0),
               dict(e0=9), dict(E=5000, e0=0, E_l=1025), dict(T=1 << 30), dict(x=None),
               dict(topk_idx=None), dict(topk_w=None), dict(y=None), dict(gate_codes=None),
               dict(down_scales=None), dict(up_codes=24), dict(down_scales=17), dict(gate_zeros=16),
               dict(down_zeros=16), dict(x=24), dict(y=20), dict(y_in=20), dict(d=(1 << 22) + 64)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(workspace=None), dict(workspace_bytes=64), dict(workspace=24)):
        assert call(**kw) == EWORKSPACE, kw
    assert call(T=0, x=None, workspace=None) == OK
    assert lib.mok_moe_w4_forward(None, None) == EINVAL
    small = [mok.mok_moe_w4_workspace_bytes(moe_args(mok, T=T)) for T in (0, 1, 100, 256, 257, 4000)]
    assert small[0] > 0 and small == sorted(small)          # a layer's workspace serves fewer tokens


def test_struct_layout_matches_header(mok, tmp_path):
    fields = [f[0] for f in mok.MoeW4Args._fields_]
    src = tmp_path / "layout.c"
    body = "".join(f'printf("%s %zu\\n", "{f}", offsetof(mok_moe_w4_args, {f}));' for f in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mok.h"\nint main(void){' + body
                   + 'printf("sizeof %zu\\n", sizeof(mok_moe_w4_args));return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    out = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    for f in fields:
        assert int(out[f]) == getattr(mok.MoeW4Args, f).offset, f
    assert int(out["sizeof"]) == ctypes.sizeof(mok.MoeW4Args)


def test_tensors_that_cannot_be_marshalled(mok):
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    b = torch.zeros(4, 64).bfloat16()
    c, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 1).bfloat16()
    c3, s3 = torch.zeros(2, 8, 32, dtype=torch.uint8), torch.zeros(2, 8, 1).bfloat16()
    calls = [
        lambda: mok.mok_topk_scored(f, 2, i, f[:, :2]),
        lambda: mok.mok_topk_scored(f, 2, i, f[:, :2], score="linear"),
        lambda: mok.mok_topk_scored(f[0], 2, i, f[:, :2]),
        lambda: mok.mok_route_scored(f, f, 2, f, i, f),
        lambda: mok.mok_topk_scored_backward(f, i, f, f),
        lambda: mok.mok_gated_norm(f, f, 1e-6, f),
        lambda: mok.mok_gated_norm(f.half(), f, 1e-6, f),
        lambda: mok.mok_gated_norm_backward(f, f, f, f),
        lambda: mok.mok_quantize_int4(b, c[:4], s[:4]),
        lambda: mok.mok_quantize_int4(b, c, s),
        lambda: mok.mok_w4_gemm(b, c, s, f),
        lambda: mok.mok_w4_gemm(b, c, s, f.half()),
        lambda: mok.MoeW4Layer((c3, s3, None), (c3, s3, None), (c3, s3, None), E=4, k=2, max_tokens=4),
        lambda: mok.MoeW4Layer((c, s, None), (c, s, None), (c, s, None), E=4, k=2, max_tokens=4),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(mok.MokError) as e:
            call()
        assert e.value.status == EINVAL, n


def test_workspace_queries(mok):
    assert mok.mok_gated_norm_backward_workspace_bytes(0, 64) > 0
    for call in (lambda: mok.mok_gated_norm_backward_workspace_bytes(-1, 8),
                 lambda: mok.mok_moe_w4_workspace_bytes(moe_args(mok, group=16))):
        with pytest.raises(mok.MokError) as e:
            call()
        assert e.value.status == EINVAL


def test_more_tokens_than_a_launch(lib):
    """Past 2^25 tokens the choice and its gradient are refused, not launched."""
    T = (1 << 25) + 1
    rule = dict(score=1, bias=None, G=4, Gk=2, top=2, renorm=1, scale=1.0)
    refuse(lib.mok_topk_scored, dict(logits=16, T=T, E=16, k=1, **rule, idx=16, w=16), EUNSUPPORTED)
    refuse(lib.mok_route_scored, dict(x=16, wr=16, T=T, d=64, E=16, k=1, io=1, **rule, logits=16, idx=16, w=16),
           EUNSUPPORTED)
    refuse(lib.mok_topk_scored_backward, dict(logits=16, idx=16, dw=16, din=None, T=T, E=16, k=1, score=0, renorm=0,
                                              scale=1.0, dl=16), EUNSUPPORTED)
    refuse(lib.mok_topk_scored, dict(logits=16, T=1 << 62, E=16, k=4, **rule, idx=16, w=16), EINVAL)
