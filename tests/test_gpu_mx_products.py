"""Microscaled product: which products are exact, and long K in every tile form.

The matrix instruction cuts the products of a 32-value block off on a grid 13 bits below the largest
sum of two exponents (subnormals counted with their type's least one): with u(v) = max(|v|, smallest
normal of v's type), 2^-6 in E4M3 and 1 in E2M1, a block loses less than 32 2^-13 = 2^-8 of the
largest u(a) u(b) among its products. With one E2M1 operand, float32 results and up to 64 rows lose
nothing."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
GRID = [0, .5, 1, 1.5, 2, 3, 4, 6]


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def table(fmt):
    """(float64 values by code, with the NaN codes at 0; smallest normal)"""
    if fmt == 4:
        v = torch.tensor(GRID, dtype=torch.float64)
        return torch.cat([v, -v]).to(DEV), 1.0
    v = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    return torch.nan_to_num(v, nan=0.0).to(DEV), 2.0 ** -6


def packed(codes, fmt):
    return codes if fmt == 8 else (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def gemm(mok, a, asc, b, bsc, dtype):
    M, N, K = a.shape[0], b.shape[0], 32 * asc.shape[1]
    n = mok.mok_mx_gemm_workspace_bytes(M, N, K)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if n else None
    c = torch.full((M, N), 7.0, dtype=dtype, device=DEV)
    mok.mok_mx_gemm(a, asc, b, bsc, c, ws)
    torch.cuda.synchronize()
    return c


def pairs(fmt, sign):
    """Rows [v, sign v, s, 0 ...] for every two positive finite values v, s: (codes, values of s)."""
    n = 7 if fmt == 4 else 126
    c = torch.arange(1, n + 1, device=DEV).to(torch.uint8)
    v, s = c.repeat_interleave(n), c.repeat(n)
    codes = torch.zeros((n * n, 32), dtype=torch.uint8, device=DEV)
    codes[:, 0], codes[:, 2] = v, s
    codes[:, 1] = v + ((8 if fmt == 4 else 0x80) if sign < 0 else 0)
    return packed(codes, fmt), table(fmt)[0][s.long()]


@pytest.mark.parametrize("fa,fb", [(8, 4), (4, 8)])
def test_float32_results_of_mixed_pairs_lose_no_product(fa, fb):
    """v t + s u - v t for every v, s and t, u: what is left is s u, to its last bit. In tiles, and
    with the E2M1 operand's 49 rows in the form of few rows."""
    import routing_grouped_expert_gemm_amd as mok
    (a, s), (b, u) = pairs(fa, 1), pairs(fb, -1)
    one = [torch.full((t.shape[0], 1), 127, dtype=torch.uint8, device=DEV) for t in (a, b)]
    ref = s[:, None] * u[None, :]
    assert torch.equal(gemm(mok, a, one[0], b, one[1], torch.float32).double(), ref)
    assert torch.equal(gemm(mok, b, one[1], a, one[0], torch.float32).double(), ref.T)


def rows(M, K, fmt, g, scales=(120, 134)):
    """Any finite codes, the larger ones more often: (codes, scales, values, their u)."""
    t, tiny = table(fmt)
    if fmt == 4:
        c = torch.randint(0, 16, (M, K), generator=g, device=DEV)
    else:
        c = torch.randint(0, 127, (M, K), generator=g, device=DEV)
        c = torch.where(torch.rand(M, K, generator=g, device=DEV) < 0.3, c % 16 + 111, c)
        c = c + 128 * torch.randint(0, 2, (M, K), generator=g, device=DEV)
    sc = torch.randint(*scales, (M, K // 32), generator=g, device=DEV)
    v = t[c]
    f = torch.exp2(sc.double() - 127)[:, :, None]
    u = torch.where(v == 0, 0.0, v.abs().clamp(min=tiny))
    return (packed(c.to(torch.uint8), fmt), sc.to(torch.uint8),
            (v.view(M, -1, 32) * f).view(M, K), (u.view(M, -1, 32) * f).view(M, K))


@pytest.mark.parametrize("fa,fb", [(4, 4), (8, 4), (4, 8), (8, 8)])
@pytest.mark.parametrize("M,N,K", [(40, 50, 32), (48, 40, 320), (90, 70, 32), (100, 70, 352), (70, 66, 2048)])
def test_any_codes_within_the_blocks_grid(M, N, K, fa, fb):
    """Every block may lose 2^-8 of its largest u(a) u(b) (nothing with an E2M1 operand and a
    float32 result or up to 64 rows); K / 32 sums in float32 and the output type's half step come on
    top. The instruction takes two blocks, whose sums are rounded, each to float32, into the
    accumulator: (K / 32 + 8) 2^-23 of sum |a b|."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator(device=DEV).manual_seed(M + N + K + fa * 3 + fb)
    (a, asc, av, au), (b, bsc, bv, bu) = rows(M, K, fa, g), rows(N, K, fb, g)
    b[1], bsc[1], bv[1], bu[1] = (t[0] for t in (b, bsc, bv, bu))
    ref, mag = torch.zeros(M, N, dtype=torch.float64, device=DEV), torch.zeros(M, N, dtype=torch.float64, device=DEV)
    lost = torch.zeros_like(ref)
    for k in range(0, K, 32):
        p = av[:, None, k:k + 32] * bv[None, :, k:k + 32]
        ref += p.sum(2)
        mag += p.abs().sum(2)
        lost += (au[:, None, k:k + 32] * bu[None, :, k:k + 32]).amax(2) * 2.0 ** -8
    sums = (K / 32 + 8) * 2.0 ** -23 * mag
    for dtype in (torch.float32, torch.bfloat16):
        exact = fa == fb == 4 or (fa != fb and (dtype is torch.float32 or M <= 64))
        got = gemm(mok, a, asc, b, bsc, dtype).double()
        tol = sums + (0.0 if exact else lost)
        if dtype is torch.bfloat16:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        assert ((got - ref).abs() <= tol).all()


@pytest.mark.parametrize("fa,fb,most", [(8, 8, 1.5e-5), (8, 4, 1e-7), (4, 8, 1e-7), (4, 4, 1e-7)])
def test_error_on_normal_rows(fa, fb, most):
    """The documented errors' norms on quantised normal rows (float32 results), and how often a
    bf16 result is not the rounded exact one: an error of 5e-6 moves it over a border of two values,
    which lie 2^-8 of it apart or more, with a chance of 5e-6 2^8 = 0.13% at the norm, and more for
    smaller results, whose steps are smaller: below 1%. (The float32 error of K / 32 sums: its random
    roundings sqrt(K / 16) 2^-24 and as much again.)"""
    import routing_grouped_expert_gemm_amd as mok
    M, N, K = 400, 320, 4096
    g = torch.Generator(device=DEV).manual_seed(fa * 10 + fb)
    ops, vals = [], []
    for n, f in ((M, fa), (N, fb)):
        x = torch.randn(n, K, generator=g, device=DEV).to(torch.bfloat16)
        c = torch.empty((n, K if f == 8 else K // 2), dtype=torch.uint8, device=DEV)
        s = torch.empty((n, K // 32), dtype=torch.uint8, device=DEV)
        (mok.mok_quantize_mxfp8 if f == 8 else mok.mok_quantize_mxfp4)(x, c, s)
        ops += [c, s]
        c = c.long() if f == 8 else torch.stack([c & 15, c >> 4], 2).view(n, K).long()
        vals.append((table(f)[0][c].view(n, -1, 32) * torch.exp2(s.double() - 127)[:, :, None]).view(n, K))
    ref = vals[0] @ vals[1].T.contiguous()
    err = gemm(mok, *ops, torch.float32).double() - ref
    assert float(err.norm() / ref.norm()) <= max(1.25 * most, 4 * (K / 16 + 8) ** 0.5 * 2.0 ** -24)
    got = gemm(mok, *ops, torch.bfloat16)
    off = float((got != ref.float().to(torch.bfloat16)).double().mean())
    assert off <= (0.03 if fa == fb == 8 else 0.01)


def exact_operand(M, K, fmt, g):
    """Codes on the E2M1 grid under scales 1 and 2: products are multiples of 1/4 of at most 144, and
    sums of up to 2^14.5 of them are below 2^24 quarters: exact in float32 in any order."""
    nib = torch.randint(0, 16, (M, K), generator=g, device=DEV)
    val = table(4)[0][nib]
    sc = torch.randint(127, 129, (M, K // 32), generator=g, device=DEV)
    if fmt == 4:
        codes = packed(nib.to(torch.uint8), 4)
    else:
        by_nib = table(4)[0].float().cpu().to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
        codes = by_nib[nib]
    return codes, sc.to(torch.uint8), (val.view(M, -1, 32) * torch.exp2(sc.double() - 127)[:, :, None]).view(M, K)


def moved(t):
    """The same bytes one past a 16-byte address."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    b[1:] = t.flatten()
    return b[1:].view(t.shape)


LONG = [  # M, N, K, scales off 16 bytes
    # 196 tiles of 256 x 256: scales by DMA in 3 and 5 groups of 32 blocks, through registers (off 16
    # bytes; K not a multiple of 512, with a ragged last step)
    (3400, 3500, 2560, False), (3400, 3520, 4608, False), (3400, 3520, 2560, True),
    (3400, 3500, 2592, False), (3390, 3520, 4128, False), (3400, 3500, 544, False),
    # 48 tiles of 128 x 128, one range of K: 6 groups of scales by DMA (they turn over four buffers)
    # and through registers
    (700, 904, 5632, False), (700, 900, 5632, True), (700, 904, 5664, False), (700, 904, 1536, False),
    # 30 tiles: 4 ranges of K of 5 and more groups each; 6 tiles: 7 and 16 ranges
    (700, 600, 20480, False), (700, 600, 20512, False), (130, 260, 7168, True), (130, 260, 16384, False),
    # up to 64 rows
    (33, 40, 20480, True), (1, 100, 20512, False)]


@pytest.mark.parametrize("fa,fb", [(4, 4), (8, 4), (4, 8), (8, 8)])
@pytest.mark.parametrize("M,N,K,off", LONG)
def test_long_k_in_every_tile_form(M, N, K, off, fa, fb):
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator(device=DEV).manual_seed(M + N + K + fa * 3 + fb)
    (a, asc, av), (b, bsc, bv) = exact_operand(M, K, fa, g), exact_operand(N, K, fb, g)
    if off:
        asc, bsc = moved(asc), moved(bsc)
    ref = av @ bv.T.contiguous()
    assert torch.equal(gemm(mok, a, asc, b, bsc, torch.float32).double(), ref)
    assert torch.equal(gemm(mok, a, asc, b, bsc, torch.bfloat16), ref.float().to(torch.bfloat16))
