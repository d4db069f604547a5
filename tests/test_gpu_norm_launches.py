"""Residual RMS norm past the rows of one launch (2^21), and rows of whole 16-byte pieces at other
addresses, which take the form of one value a step.

Tolerances: those of the norm's tests, u = 2^-24: y and rstd off by 64 u of themselves (128 u at other
addresses) and half a step of the type, dx by 128 u (256 u) of its absolute terms and half a step. dweight
adds rows / 512 rows in a chain, then 512 sums in chains of 8 and a tree: (rows / 512 + 80) u of sum |dy n|."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def off(t):
    """The same values one behind a 16-byte address."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    b[1:] = t.flatten()
    return b[1:].view(t.shape)


def check(mok, T, d, dtype, at, wide, codes):
    t = TYPES[dtype]
    half = 0.0 if t is torch.float32 else torch.finfo(t).eps / 2
    g = torch.Generator(device=DEV).manual_seed(T + d)
    x, res, dy, dh = (at(torch.randn(T, d, generator=g, device=DEV).to(t)) for _ in range(4))
    w = at((1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t))
    h, y, dx = (at(torch.full((T, d), 7.0, dtype=t, device=DEV)) for _ in range(3))
    rstd, dw = torch.full((T,), 7.0, device=DEV), torch.full((d,), 7.0, device=DEV)
    q = at(torch.full((T, d), 0xEE, dtype=torch.uint8, device=DEV)) if codes else None
    s = torch.full((T, d // 32), 0xEE, dtype=torch.uint8, device=DEV) if codes else None
    ws = torch.empty(mok.mok_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    mok.mok_rmsnorm(x, w, EPS, residual=res, h=h, y=y, rstd=rstd, codes=q, scales=s)
    mok.mok_rmsnorm_backward(dy, h, rstd, w, dx, dw, ws, dh=dh)
    torch.cuda.synchronize()
    assert torch.equal(h, x + res)
    v, wt, gy = h.double(), w.double(), dy.double()
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    n, gw = v * r, gy * wt
    assert ((rstd.double()[:, None] - r).abs() <= wide * 64 * U * r).all()
    ref = n * wt
    assert ((y.double() - ref).abs() <= (wide * 64 * U + half) * ref.abs() + 1e-37).all()
    if codes:                                  # those of the quantiser, as float32 y is rounded once
        yf = torch.empty(T, d, device=DEV)
        mok.mok_rmsnorm(h.float(), w.float(), EPS, y=yf)
        q2, s2 = torch.empty((T, d), dtype=torch.uint8, device=DEV), torch.empty_like(s)
        mok.mok_quantize_mxfp8_f32(yf, q2, s2)
        torch.cuda.synchronize()
        assert torch.equal(q, q2) and torch.equal(s, s2)
    m = (gw * n).mean(1, keepdim=True)
    ref = r * (gw - n * m) + dh.double()
    mag = r * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True)) + dh.double().abs()
    assert ((dx.double() - ref).abs() <= wide * 128 * U * mag + half * ref.abs() + 1e-37).all()
    ref, mag = (gy * n).sum(0), (gy * n).abs().sum(0)
    assert ((dw.double() - ref).abs() <= (T / 512 + 80) * U * mag).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [((1 << 21) + 1, 8), ((1 << 22) + 777, 8), ((1 << 21) + 3, 3), ((1 << 22) + 5, 1),
                                 ((1 << 21) + 70, 32)])
def test_more_rows_than_a_launch(T, d, dtype):
    import routing_grouped_expert_gemm_amd as mok
    check(mok, T, d, dtype, lambda t: t, 2 if d % 8 else 1, d == 32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(5, 8), (300, 64), (9, 2048), (700, 4096), (3, 8192)])
def test_whole_pieces_at_any_address(T, d, dtype):
    import routing_grouped_expert_gemm_amd as mok
    check(mok, T, d, dtype, off, 2, d % 32 == 0)
