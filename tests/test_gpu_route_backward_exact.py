"""Router backward on inputs whose sums are exact in float32 in any order, so that the outputs have to
be equal to the definition's: one token, range or tile left out or counted twice shows.

Routing weights are 1 / k, k a power of two, and dtopk_w multiples of k k, so that the picks' share of
dl is made of integers. "small": dl of at most 25, x of -1, 0, 1: sums over T tokens stay below
25 T < 2^24. "fine": dlogits of 257 or -257 (two bf16 values) in up to a fourth of the tokens, where x
is not zero: below 282 T / 4 < 2^24. "planes": 65,793 (three bf16 values) in 200 tokens, the first and
the last ones among them: below 65,818 x 200 < 2^24. dx's sums over E experts, of at most (dl |W|) with
|W| 1 in up to 60 of them, stay below 2^24 as well ("planes": not compared for bf16, where dx takes 16
bits of dl)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def inputs(T, d, E, dtype, kind, seed=0):
    g = torch.Generator(device=DEV).manual_seed(T * 13 + d * 7 + E + seed)
    t, k = TYPES[dtype], 4 if E >= 4 else 1

    def pick(values, *shape):
        v = torch.tensor(values, device=DEV, dtype=torch.float32)
        return v[torch.randint(0, len(values), shape, generator=g, device=DEV)]

    x = pick([-1, 0, 1], T, d)
    dl = pick([-1, 0, 1], T, E)
    if kind != "small":
        keep = torch.zeros(T, 1, device=DEV)
        if kind == "fine":
            keep[::4] = 1
        else:
            keep[torch.randint(0, T, (150,), generator=g, device=DEV)] = 1
            keep[:10], keep[-30:] = 1, 1
        x *= keep
        dl *= 257 if kind == "fine" else 65793
    w = pick([-1, 0, 1], E, d)
    for e0 in range(60, E, 60):                   # 60 experts of a column at most
        w[e0:e0 + 60] *= (torch.arange(d, device=DEV) % (E // 60 + 1) == e0 // 60).float()
    if E > 60:
        w[:60] *= (torch.arange(d, device=DEV) % (E // 60 + 1) == 0).float()
    return dict(x=x.to(t), w=w.to(t), idx=torch.randint(0, E, (T, k), generator=g, device=DEV).int(),
                tw=torch.full((T, k), 1.0 / k, device=DEV), dtw=pick([-k * k, 0, k * k], T, k),
                dl=dl, dx_in=pick([-2, -1, 0, 1, 2], T, d).to(t))


def definition(i):
    tw, dtw = i["tw"].double(), i["dtw"].double()
    g = tw * (dtw - (tw * dtw).sum(1, keepdim=True))
    dl = i["dl"].double().scatter_add(1, i["idx"].long(), g)
    return (dl @ i["w"].double() + i["dx_in"].double()).to(i["x"].dtype), \
        dl.T.contiguous() @ i["x"].double()


def run(mok, i, dx_in=True, dlogits=True, dtw=None):
    (T, d), E = i["x"].shape, i["w"].shape[0]
    dx, dw = torch.full_like(i["x"], 7.0), torch.full((E, d), 7.0, device=DEV)
    ws = torch.full((mok.mok_route_backward_workspace_bytes(T, d, E, i["x"].dtype),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    mok.mok_route_backward(i["x"], i["w"], i["idx"], i["tw"], i["dtw"] if dtw is None else dtw, dx, dw,
                           ws, dlogits=i["dl"] if dlogits else None, dx_in=i["dx_in"] if dx_in else None)
    torch.cuda.synchronize()
    return dx, dw


CASES = [  # T, d, E
    # few experts
    (2100, 2003, 7), (70000, 61, 5), (4195000, 1, 1), (1100, 4001, 16), (16383, 257, 1), (40001, 129, 4),
    # 9 to 16 experts, narrow and wider rows
    (70001, 61, 16), (40000, 128, 9), (40001, 129, 16),
    # the plane form, tiles of 128 and 256 columns, rows that are copied
    (8192, 512, 64), (8190, 520, 130), (98300, 8, 64), (16500, 1416, 20), (16400, 1288, 130),
    (98300, 11, 64), (33000, 3, 1000), (16500, 1417, 20), (16400, 1283, 130), (1030, 1020, 64),
    # the any-size form (float32; small bf16 rows)
    (5000, 40, 8), (16500, 177, 20), (3000, 50, 30), (4097, 97, 260), (700, 33, 1024)]


@pytest.mark.parametrize("kind", ["small", "fine", "planes"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d,E", CASES)
def test_equal_to_the_definition(T, d, E, dtype, kind):
    import routing_grouped_expert_gemm_amd as mok
    if kind == "fine" and T * 282 // 4 >= 1 << 24:
        kind = "planes"
    i = inputs(T, d, E, dtype, kind)
    dx, dw = run(mok, i)
    rx, rw = definition(i)
    assert torch.equal(dw.double(), rw)
    if kind != "planes" or dtype == "fp32":
        assert torch.equal(dx, rx)
