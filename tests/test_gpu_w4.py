"""4-bit weights in groups (mok_quantize_int4, mok_w4_gemm) and the experts' FFNs on them
(mok_moe_w4_forward, MoeW4Layer) against float64.

Tolerances, u = 2^-24. A product's terms x q and -x z are exact; an MFMA adds 32 of each to a float32
sum, so a group's chain has at most 8 roundings of sums no larger than A = sum |x| (q + z), scaled and
added over at most K / 32 groups and 8 waves. Taken as 2 roundings an MFMA: (2 (K / 32) + 64) u of
sum_groups s A covers it (the instruction's own cut of aligned products is counted as one rounding).
The experts' layer: H's products as above for gate and up, silu with the hardware's exponential and
reciprocal (8 u), H enters as 16 bits (2^-17), the rest as above; an error of gate g moves silu(g) by at
most 1.1 of it.
Up to 4 rows are integers: a value of x (or H) is off by at most 2^-22 of its group's largest. bf16 values
within 2^-14 of that are exact, and the random ones here are, but for a few whose 2^-22 the bound's 64 u
of the whole sum covers many times over; where it might not (test_magnitudes) the term is in the bound. For H
the 2^-17 of each value covers it while a group's mean is above 1 / 32 of its largest. Outputs are off by half a step of their type besides (bf16: 2^-8 of the value)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def weight(g, lead, N, K, group, zeros, scale=1.0):
    c = torch.randint(0, 256, (*lead, N, K // 2), generator=g, dtype=torch.uint8)
    s = ((torch.rand((*lead, N, K // group), generator=g) + 0.5) * scale).to(torch.bfloat16)
    z = torch.randint(0, 16, s.shape, generator=g, dtype=torch.uint8) if zeros else None
    return c, s, z


def parts(w, group):
    """Codes and zero points as numbers [.., K], scales repeated."""
    c, s, z = w
    q = torch.stack([c & 15, c >> 4], -1).flatten(-2).double().numpy()
    r = lambda t: t.double().repeat_interleave(group, -1).numpy()  # noqa: E731
    return q, (np.full(q.shape, 8.0) if z is None else r(z)), r(s)


def dense(w, group):
    q, z, s = parts(w, group)
    return (q - z) * s, (q + z) * np.abs(s)


def product(x, w, group):
    """x W^T and its bound."""
    W, A = dense(w, group)
    K = W.shape[-1]
    return x @ W.T, (2 * (K / 32) + 64) * U * (np.abs(x) @ A.T)


def dev(w):
    return tuple(None if t is None else t.to(DEV) for t in w)


GEMMS = [(1, 1, 32, 32), (1, 16, 128, 128), (3, 17, 64, 64), (2, 33, 96, 32), (5, 100, 384, 128), (16, 48, 512, 64),
         (17, 31, 640, 128), (1, 257, 1408, 128), (8, 64, 1056, 32), (13, 130, 2048, 64), (64, 64, 192, 64), (33, 20, 4096, 128),
         (7, 40, 4224, 128), (4, 24, 4160, 64), (9, 50, 7168, 128), (2, 30, 7168, 32), (1, 19, 8320, 128), (16, 16, 9000 // 64 * 64, 64),
         (3, 5, 16384 + 128, 128), (6, 9, 12288 + 32, 32), (130, 7, 256, 64), (1, 5000, 256, 128), (1, 40000, 64, 64)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,group", GEMMS)
def test_product(M, N, K, group, out, zeros):
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(M * 131 + N + K)
    x = (torch.randn(M, K, generator=g) + 0.3).bfloat16()
    w = weight(g, (), N, K, group, zeros)
    ref, tol = product(x.double().numpy(), w, group)
    D = dev(w)
    buf = torch.full((M * N + 64,), 7.0, dtype=out, device=DEV)
    c = buf[:M * N].view(M, N)
    mok.mok_w4_gemm(x.to(DEV), D[0], D[1], c, zeros=D[2])
    torch.cuda.synchronize()
    assert (np.abs(c.double().cpu().numpy() - ref) <= tol + half_step(out) * np.abs(ref)).all()
    assert (buf[M * N:] == 7).all()
    c2 = torch.empty_like(c)
    mok.mok_w4_gemm(x.to(DEV), D[0], D[1], c2, zeros=D[2])
    torch.cuda.synchronize()
    assert torch.equal(c, c2)


def test_product_of_whole_numbers_is_exact():
    """Inputs whose sums are exact: every position of K, and each code, zero point and group counts once."""
    import routing_grouped_expert_gemm_amd as mok
    for K, group in ((128, 32), (2048, 64), (4096, 128), (7168, 128), (8192 + 256, 64)):
        g = torch.Generator().manual_seed(K)
        N, M = 37, 16
        x = torch.randint(-3, 4, (M, K), generator=g).bfloat16()
        c, s, z = weight(g, (), N, K, group, True)
        s = torch.randint(0, 3, s.shape, generator=g).to(torch.bfloat16)
        W, _ = dense((c, s, z), group)
        out = torch.empty(M, N, device=DEV)
        mok.mok_w4_gemm(x.to(DEV), c.to(DEV), s.to(DEV), out, zeros=z.to(DEV))
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), x.double().numpy() @ W.T)


def test_rows_do_not_meet():
    """An infinite or NaN row stays alone; a weight row with a NaN scale gives a NaN column."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(1)
    M, N, K = 20, 48, 1024
    x = torch.randn(M, K, generator=g).bfloat16()
    w = weight(g, (), N, K, 128, False)
    ref, tol = product(x.double().numpy(), w, 128)
    x[3, 5], x[18, 1000] = float("inf"), float("nan")
    w[1][7, 2] = float("nan")
    out = torch.empty(M, N, device=DEV)
    mok.mok_w4_gemm(x.to(DEV), w[0].to(DEV), w[1].to(DEV), out)
    torch.cuda.synchronize()
    o = out.double().cpu().numpy()
    assert not np.isfinite(o[3]).any() and np.isnan(o[18]).all() and np.isnan(o[:, 7]).all()
    rows, cols = [r for r in range(M) if r not in (3, 18)], [c for c in range(N) if c != 7]
    assert (np.abs(o - ref)[np.ix_(rows, cols)] <= (tol + half_step(torch.float32) * np.abs(ref))[np.ix_(rows, cols)]).all()


def test_weight_past_32_bits():
    """Codes past 2^31 bytes: the last rows."""
    import routing_grouped_expert_gemm_amd as mok
    N, K, group = (1 << 31) // 4096 + 100, 8192, 128
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.ones(N, K // group, dtype=torch.bfloat16, device=DEV)
    codes[-1], codes[-50] = 0x9A, 0x11
    x = torch.ones(1, K, device=DEV).bfloat16()
    out = torch.empty(1, N, device=DEV)
    mok.mok_w4_gemm(x, codes, scales, out)
    torch.cuda.synchronize()
    assert out[0, -1] == K * 1.5 and out[0, -50] == -7 * K and (out[0, :-50] == -8 * K).all()


# ------------------------------------------------------------------------------- quantiser

def quantised(w, group, zeros):
    f = np.float32
    v = w.float().numpy().reshape(w.shape[0], -1, group)
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a)).bfloat16()  # noqa: E731
    hi, lo = np.maximum(v.max(2), f(0)), np.minimum(v.min(2), f(0))
    s = bf(hi / f(15) - lo / f(15)) if zeros else bf(np.maximum(hi, -lo) / f(7))
    sf = s.float().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(sf > 0, np.clip(np.rint(-lo / sf), 0, 15), 0) if zeros else np.full(sf.shape, 8)
        q = np.where(sf[:, :, None] > 0, np.clip(np.rint(v / sf[:, :, None]) + z[:, :, None], 0, 15), z[:, :, None])
    q = q.reshape(w.shape[0], -1).astype(np.uint8)
    return q[:, 0::2] | (q[:, 1::2] << 4), s, z.astype(np.uint8)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantiser(group, zeros):
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(group)
    for rows, K in ((1, group), (7, 3 * group), (130, 8 * group)):
        w = (torch.randn(rows, K, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))).bfloat16()
        if rows > 1:
            w[0, :group] = 0
            w[1] = w[1].abs() + 1                        # one sign: the range starts at 0
            w[2] = -w[2].abs() - 1
            w[3, :group] = 1e-38
            w[4, :group] = 0
            w[4, 3] = 1e-40                              # a scale that is subnormal or 0
            w[5, :group] *= 3e38 / w[5, :group].abs().max()
        codes = torch.full((rows, K // 2), 0xEE, dtype=torch.uint8, device=DEV)
        s = torch.full((rows, K // group), 7.0, dtype=torch.bfloat16, device=DEV)
        z = torch.full((rows, K // group), 99, dtype=torch.uint8, device=DEV) if zeros else None
        mok.mok_quantize_int4(w.to(DEV), codes, s, z)
        torch.cuda.synchronize()
        rc, rs, rz = quantised(w, group, zeros)
        assert torch.equal(s.cpu(), rs) and np.array_equal(codes.cpu().numpy(), rc)
        assert z is None or np.array_equal(z.cpu().numpy(), rz)
        # no value is further off than its half step, the scale's rounding over the codes and a clamp allow
        q, zp, sc = parts((codes.cpu(), s.cpu(), None if z is None else z.cpu()), group)
        ok = sc > 1e-36
        assert (np.abs((q - zp) * sc - w.double().numpy())[ok] <= (sc * (0.5 + 0.5 * zeros + 15 * 2.0 ** -8))[ok]).all()


def test_quantiser_marks_what_is_no_number():
    import routing_grouped_expert_gemm_amd as mok
    w = torch.ones(4, 64).bfloat16()
    w[1, 3], w[2, 40], w[3, 63] = float("nan"), float("inf"), -float("inf")
    for zeros in (False, True):
        codes, s = torch.empty(4, 32, dtype=torch.uint8, device=DEV), torch.empty(4, 2, device=DEV).bfloat16()
        z = torch.empty(4, 2, dtype=torch.uint8, device=DEV) if zeros else None
        mok.mok_quantize_int4(w.to(DEV), codes, s, z)
        torch.cuda.synchronize()
        assert torch.isnan(s.cpu()).tolist() == [[False, False], [True, False], [False, True], [False, True]]


# ------------------------------------------------------------------------------- experts

def layer_weights(g, E_l, d, I, group, zeros):
    return dict(gate=weight(g, (E_l,), I, d, group, zeros, 0.2 * d ** -0.5),
                up=weight(g, (E_l,), I, d, group, zeros, 0.2 * d ** -0.5),
                down=weight(g, (E_l,), d, I, group, zeros, 0.2 * I ** -0.5))


def moe(x, idx, tw, L, e0, group, y_in):
    """The layer in float64 and its bound before the last rounding."""
    xd = x.double().numpy()
    y = np.zeros_like(xd) if y_in is None else y_in.double().numpy().copy()
    tol = 8 * U * np.abs(y)
    E_l = L["gate"][0].shape[0]
    for e in range(E_l):
        t, j = np.nonzero(idx == e + e0)
        if not len(t):
            continue
        w = {n: tuple(None if v is None else v[e] for v in L[n]) for n in L}
        g, gt = product(xd[t], w["gate"], group)
        u, ut = product(xd[t], w["up"], group)
        sg = g / (1 + np.exp(-g))
        h = sg * u
        ht = 1.1 * gt * (np.abs(u) + ut) + np.abs(sg) * ut + (8 * U + 2.0 ** -17) * np.abs(h)
        p, pt = product(h, w["down"], group)
        _, A = dense(w["down"], group)
        Wd = np.abs(dense(w["down"], group)[0])
        pt = pt + ht @ Wd.T
        c = tw[t, j].astype(np.float64)[:, None]
        np.add.at(y, t, c * p)
        np.add.at(tol, t, np.abs(c) * (pt + 16 * U * np.abs(p)))
    return y, tol


def routing(rng, T, E, k):
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    tw = rng.random((T, k)).astype(np.float32)
    return idx, tw / tw.sum(1, keepdims=True)


LAYERS = [  # T, d, I, E, e0, E_l, k, group
    (1, 32, 32, 1, 0, 1, 1, 32), (1, 256, 128, 8, 0, 8, 2, 128), (1, 2048, 1408, 16, 0, 16, 6, 128), (3, 192, 64, 16, 0, 16, 4, 64),
    (5, 384, 256, 6, 0, 6, 3, 128), (2, 96, 160, 64, 0, 64, 8, 32), (40, 256, 128, 4, 0, 4, 2, 64), (7, 256, 192, 32, 8, 5, 8, 64),
    (64, 128, 128, 8, 0, 8, 2, 32), (130, 128, 64, 16, 3, 9, 8, 64), (128, 64, 64, 8, 0, 8, 8, 32), (129, 64, 64, 8, 0, 8, 8, 32),
    (700, 128, 96, 4, 0, 4, 3, 32), (1, 7168, 256, 4, 0, 4, 2, 128), (2, 8192 + 128, 128, 3, 0, 3, 2, 128), (2, 128, 4224, 3, 0, 3, 2, 128),
    (9, 64, 7168, 3, 1, 2, 2, 64), (20, 256, 128, 1, 0, 1, 1, 128), (16, 128, 128, 256, 0, 256, 4, 64)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,d,I,E,e0,E_l,k,group", LAYERS)
def test_experts(T, d, I, E, e0, E_l, k, group, zeros):
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(T * 7 + d + I)
    rng = np.random.default_rng(T + d)
    L = layer_weights(g, E_l, d, I, group, zeros)
    x, y_in = torch.randn(T, d, generator=g).bfloat16(), torch.randn(T, d, generator=g).bfloat16()
    idx, tw = routing(rng, T, E, k)
    if T > 4:                                            # ids of nobody, and an expert named twice
        idx[0, 0], idx[1, 0], idx[2, :] = -1, E + 3, e0
        idx[3, :] = -5
    layer = mok.MoeW4Layer(*(dev(L[n]) for n in ("gate", "up", "down")), E=E, k=k, e0=e0, max_tokens=T + 3)
    layer.workspace.fill_(0xFF)                          # NaN wherever something unwritten is read
    ix, w = torch.from_numpy(idx).to(DEV), torch.from_numpy(tw).to(DEV)
    for yi in (None, y_in):
        ref, tol = moe(x, idx, tw, L, e0, group, yi)
        buf = torch.full((T * d + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
        y = buf[:T * d].view(T, d)
        layer.forward(x.to(DEV), ix, w, y, y_in=None if yi is None else yi.to(DEV))
        torch.cuda.synchronize()
        off = np.abs(y.double().cpu().numpy() - ref) - (tol + half_step(torch.bfloat16) * np.abs(ref))
        assert (off <= 0).all(), off.max()
        assert (buf[T * d:] == 7).all()
    y2 = y_in.to(DEV)
    layer.forward(x.to(DEV), ix, w, y2, y_in=y2)         # in place
    y3 = x.to(DEV)
    layer.forward(y3, ix, w, y3, y_in=y_in.to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3)


def test_shares_add_up():
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(4)
    T, d, I, E, k, group = 11, 256, 128, 12, 4, 64
    L = layer_weights(g, E, d, I, group, True)
    x = torch.randn(T, d, generator=g).bfloat16()
    idx, tw = routing(np.random.default_rng(0), T, E, k)
    total = np.zeros((T, d))
    for e0, n in ((0, 5), (5, 1), (6, 6)):
        part = {m: tuple(v[e0:e0 + n].contiguous() for v in L[m]) for m in L}
        layer = mok.MoeW4Layer(*(dev(part[m]) for m in ("gate", "up", "down")), E=E, k=k, e0=e0, max_tokens=T)
        y = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
        layer.forward(x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(tw).to(DEV), y)
        torch.cuda.synchronize()
        total += y.double().cpu().numpy()
    ref, tol = moe(x, idx, tw, L, 0, group, None)
    size = sum(np.abs(moe(x, idx, tw, {m: tuple(v[a:b] for v in L[m]) for m in L}, a, group, None)[0])
               for a, b in ((0, 5), (5, 6), (6, 12)))
    assert (np.abs(total - ref) <= tol + half_step(torch.bfloat16) * size).all()


def test_no_tokens_and_fewer_than_before():
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(6)
    d, I, E, k, group = 128, 64, 8, 2, 32
    L = layer_weights(g, E, d, I, group, False)
    layer = mok.MoeW4Layer(*(dev(L[m]) for m in ("gate", "up", "down")), E=E, k=k, max_tokens=600)
    e = torch.empty(0, d, dtype=torch.bfloat16, device=DEV)
    layer.forward(e, torch.empty(0, k, dtype=torch.int32, device=DEV), torch.empty(0, k, device=DEV), e)
    for T in (600, 1, 513, 7, 512):
        x = torch.randn(T, d, generator=g).bfloat16()
        idx, tw = routing(np.random.default_rng(T), T, E, k)
        y = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
        layer.forward(x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(tw).to(DEV), y)
        torch.cuda.synchronize()
        ref, tol = moe(x, idx, tw, L, 0, group, None)
        assert (np.abs(y.double().cpu().numpy() - ref) <= tol + half_step(torch.bfloat16) * np.abs(ref)).all()


@pytest.mark.parametrize("T", [1, 6, 300])
def test_captured_and_replayed(T):
    """The layer and a product in one graph; another graph of the same layer in between."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(9)
    d, I, E, k, group = 512, 256, 16, 4, 128
    L = layer_weights(g, E, d, I, group, True)
    layer = mok.MoeW4Layer(*(dev(L[m]) for m in ("gate", "up", "down")), E=E, k=k, max_tokens=T)
    wo = dev(weight(g, (), 320, d, group, False))
    x = torch.randn(T, d, device=DEV).bfloat16()
    idx, tw = torch.zeros(T, k, dtype=torch.int32, device=DEV), torch.rand(T, k, device=DEV)
    mk = lambda: (torch.empty_like(x), torch.empty(T, 320, device=DEV))  # noqa: E731

    def go(y, o):
        layer.forward(x, idx, tw, y)
        mok.mok_w4_gemm(y, wo[0], wo[1], o)

    def draw():
        x.normal_()
        idx.copy_(torch.rand(T, E, device=DEV).topk(k).indices)

    draw()
    a, b, e = mk(), mk(), mk()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(*a)
    torch.cuda.synchronize()
    graphs = []
    for o in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            go(*o)
    for i in range(4):
        draw()
        for q in graphs:
            q.replay()
        torch.cuda.synchronize()
        go(*e)
        torch.cuda.synchronize()
        for o in (a, b):
            assert torch.equal(o[0], e[0]) and torch.equal(o[1], e[1]), i


# ------------------------------------------------------------------------------- forms

@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", [(13, 4120, 1152, 128), (6, 4200, 416, 32), (40, 2100, 192, 64), (16, 4128, 4224, 128),
                                         (5, 8200, 2112, 64), (16, 4096, 1024, 32), (16, 4097, 1024, 32)])
def test_product_of_many_tiles(M, N, K, group, zeros):
    test_product(M, N, K, group, torch.float32, zeros)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,d,I,E,e0,E_l,k,group", [
    (1, 64, 4224, 32, 0, 32, 8, 32), (2, 192, 8320, 24, 0, 24, 3, 64), (1, 96, 4128, 8, 0, 8, 1, 32), (1, 128, 128, 36, 0, 36, 9, 128),
    (8, 256, 1152, 128, 0, 128, 4, 128), (5, 256, 128, 160, 0, 160, 8, 64), (1, 4096, 512, 40, 0, 40, 5, 128)])
def test_experts_of_lone_tokens(T, d, I, E, e0, E_l, k, group, zeros):
    test_experts(T, d, I, E, e0, E_l, k, group, zeros)


def test_tokens_of_one_expert():
    """Every token of the batch picks the same experts, where hardly any was expected to."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(12)
    T, d, I, E, k, group = 12, 256, 384, 256, 4, 128
    L = layer_weights(g, E, d, I, group, True)
    layer = mok.MoeW4Layer(*(dev(L[m]) for m in ("gate", "up", "down")), E=E, k=k, max_tokens=T)
    x = torch.randn(T, d, generator=g).bfloat16()
    idx, tw = routing(np.random.default_rng(5), T, E, k)
    for rows in (np.tile(idx[:1], (T, 1)), np.full((T, k), 255, np.int32)):
        y = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
        layer.forward(x.to(DEV), torch.from_numpy(rows).to(DEV), torch.from_numpy(tw).to(DEV), y)
        torch.cuda.synchronize()
        ref, tol = moe(x, rows, tw, L, 0, group, None)
        assert (np.abs(y.double().cpu().numpy() - ref) <= tol + half_step(torch.bfloat16) * np.abs(ref)).all()


@pytest.mark.parametrize("M", [1, 4, 7])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_magnitudes(M, group):
    """Groups of x from 2^-100 to 2^60 with values over 30 binades in each, zero and subnormal groups: the bound of
    test_product, and 2^-22 of a group's largest value times its codes. 1e-30: scales times what is subnormal."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(M + group)
    N, K = 40, 1024
    x = torch.randn(M, K // group, group, generator=g).double()
    x *= torch.exp2(torch.randint(-30, 1, x.shape, generator=g).double())
    x *= torch.exp2(torch.randint(-100, 61, (M, K // group, 1), generator=g).double())
    x[:, 1], x[:, 2] = 0, 1e-39
    x = x.reshape(M, K).bfloat16()
    w = weight(g, (), N, K, group, True)
    xd = x.double().numpy()
    ref, tol = product(xd, w, group)
    W, _ = dense(w, group)
    lost = 2.0 ** -22 * np.abs(xd).reshape(M, -1, group).max(2).repeat(group, 1)
    tol = tol + lost @ np.abs(W).T + 1e-30
    D = dev(w)
    out = torch.empty(M, N, device=DEV)
    mok.mok_w4_gemm(x.to(DEV), D[0], D[1], out, zeros=D[2])
    torch.cuda.synchronize()
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol + half_step(torch.float32) * np.abs(ref)).all()


def test_most_rows():
    import routing_grouped_expert_gemm_amd as mok
    M, N, K = 1 << 20, 16, 32
    x = torch.zeros(M, K, device=DEV).bfloat16()
    x[:, 0] = (torch.arange(M, device=DEV) % 200).bfloat16()
    codes = torch.full((N, K // 2), 0x9A, dtype=torch.uint8, device=DEV)       # 2, then 1
    scales = torch.ones(N, 1, device=DEV).bfloat16()
    out = torch.empty(M, N, device=DEV)
    mok.mok_w4_gemm(x, codes, scales, out)
    torch.cuda.synchronize()
    assert torch.equal(out, (2 * x[:, :1].float()).expand(M, N))


def test_two_streams_and_two_layers():
    """Two layers of the same weights, each with its workspace, run at once on two streams."""
    import routing_grouped_expert_gemm_amd as mok
    g = torch.Generator().manual_seed(3)
    T, d, I, E, k, group = 9, 1024, 512, 16, 4, 64
    L = layer_weights(g, E, d, I, group, False)
    W = [dev(L[m]) for m in ("gate", "up", "down")]
    layers = [mok.MoeW4Layer(*W, E=E, k=k, max_tokens=T) for _ in range(2)]
    xs = [torch.randn(T, d, generator=g).bfloat16().to(DEV) for _ in range(2)]
    routes = [routing(np.random.default_rng(i), T, E, k) for i in range(2)]
    ix = [(torch.from_numpy(a).to(DEV), torch.from_numpy(b).to(DEV)) for a, b in routes]
    want = []
    for i in range(2):
        want.append(torch.empty(T, d, dtype=torch.bfloat16, device=DEV))
        layers[i].forward(xs[i], *ix[i], want[i])
    torch.cuda.synchronize()
    got = [torch.empty_like(v) for v in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                layers[i].forward(xs[i], *ix[i], got[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
