"""Measured cases of the operators that complete the block around the MoE layer: the router's rule
(scores, balance bias, groups, renormalised weights) with its gradient, products with 4-bit weights
in groups, the experts' FFNs on such weights for a few tokens, and the gated norm that joins a
block's output to the residual stream, with its backward.

Each case runs in two forms on the same inputs: `own` false computes the operator in elementary
torch operations in float32 (the choice of experts in float64, whose borders decide integers),
`own` true through the library's entry points. `exact` gives the same outputs from the definitions
in float64.
"""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-6          # of the norms

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # choice of experts from a router's logits
        # one token of decoding: 256 experts in 8 groups, sigmoid scores with a balance bias
        {"name": "route_t1_e256_groups", "op": "route", "train": False, "T": 1, "E": 256, "k": 8,
         "score": "sigmoid", "bias": True, "G": 8, "Gk": 4, "top": 2, "renorm": True,
         "scale": 2.5},
        # training, one batch of the 64-expert layer: softmax scores used as they are
        {"name": "route_train_t8192_e64", "op": "route", "train": True, "T": 8192, "E": 64, "k": 6,
         "score": "softmax", "bias": False, "G": 1, "Gk": 1, "top": 1, "renorm": False,
         "scale": 1.0},
        # training, a token pool over 256 experts in groups
        {"name": "route_train_t65536_e256_groups", "op": "route", "train": True, "T": 65536,
         "E": 256, "k": 8, "score": "sigmoid", "bias": True, "G": 8, "Gk": 4, "top": 2,
         "renorm": True, "scale": 2.5},
        # products with a 4-bit weight
        # one token through a down projection, groups of 128
        {"name": "w4_t1_n7168_k2048", "op": "w4", "M": 1, "N": 7168, "K": 2048, "g": 128,
         "zeros": False, "out": "bf16"},
        # a ragged batch of decoding tokens, groups of 32 with zero points, float32 results
        {"name": "w4_t13_n4096_k7168_g32", "op": "w4", "M": 13, "N": 4096, "K": 7168, "g": 32,
         "zeros": True, "out": "fp32"},
        # the experts' FFNs on 4-bit weights
        # one token of the 64-expert layer
        {"name": "moe_w4_t1_d2048_e64", "op": "moe", "T": 1, "d": 2048, "I": 1408, "E": 64,
         "e0": 0, "El": 64, "k": 6, "g": 128, "zeros": False},
        # one token of the 256-expert layer, all experts on this GPU
        {"name": "moe_w4_t1_d7168_e256", "op": "moe", "T": 1, "d": 7168, "I": 2048, "E": 256,
         "e0": 0, "El": 256, "k": 8, "g": 128, "zeros": False},
        # a decoding batch of 48 tokens on one of eight ranks of that layer, with zero points
        {"name": "moe_w4_t48_d7168_e32of256", "op": "moe", "T": 48, "d": 7168, "I": 2048,
         "E": 256, "e0": 96, "El": 32, "k": 8, "g": 64, "zeros": True},
        # block output -> norm -> gate -> residual stream -> norm
        # one token of decoding
        {"name": "gnorm_t1_d7168", "op": "gnorm", "train": False, "T": 1, "d": 7168,
         "dtype": "bf16", "gate": "row", "post": True, "pre": True},
        # a prompt
        {"name": "gnorm_t8192_d7168", "op": "gnorm", "train": False, "T": 8192, "d": 7168,
         "dtype": "bf16", "gate": "all", "post": True, "pre": True},
        # training, one batch, a gate value for every element
        {"name": "gnorm_train_t8192_d2048", "op": "gnorm", "train": True, "T": 8192, "d": 2048,
         "dtype": "bf16", "gate": "row", "post": True, "pre": True},
        # training in float32, odd sizes, one gate for all tokens
        {"name": "gnorm_train_fp32_t1001_d1111", "op": "gnorm", "train": True, "T": 1001,
         "d": 1111, "dtype": "fp32", "gate": "all", "post": True, "pre": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "w4", "moe", "gnorm"])
    if op == "route":
        G = rng.choice([1, 1, 2, 3, 4, 8])
        E = G * _log_int(rng, 4, 512 // G)
        train = rng.random() < 0.5
        T = max(1, min(_log_int(rng, 1, 65536), 65536 * 256 // E))
        Gk = rng.randint(1, G)
        return {"op": op, "train": train, "T": T, "E": E,
                "k": rng.randint(1, min(8, E // G * Gk)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6, "G": G,
                "Gk": Gk, "top": rng.randint(1, 2), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5])}
    if op == "w4":
        g = rng.choice([32, 64, 128])
        return {"op": op, "M": _log_int(rng, 1, 64), "N": _log_int(rng, 16, 7168),
                "K": g * _log_int(rng, 1, 7168 // g), "g": g, "zeros": rng.random() < 0.5,
                "out": "bf16" if rng.random() < 0.7 else "fp32"}
    if op == "moe":
        g = rng.choice([32, 64, 128])
        d, I = g * _log_int(rng, 2, 7168 // g), g * _log_int(rng, 1, 2048 // g)
        E = _log_int(rng, 4, 256)
        El = E if rng.random() < 0.5 else rng.randint(1, E)
        k = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 48)
        El = max(1, min(El, 256 * 7168 * 2048 // (d * I)))
        ffns = max(1, 32 * 7168 * 2048 // (d * I))       # no more FFNs than the largest case
        if T * k <= El:
            T = max(1, min(T, ffns // k))
        else:                  # the plain form then runs every local expert on all tokens
            El = min(El, ffns)
        return {"op": op, "T": T, "d": d, "I": I, "E": E, "e0": rng.randint(0, E - El), "El": El,
                "k": k, "g": g, "zeros": rng.random() < 0.5}
    train = rng.random() < 0.5
    d = _log_int(rng, 32, 8192)
    if rng.random() < 0.7:
        d = d // 8 * 8
    T = max(1, min(_log_int(rng, 1, 16384), 8192 * (2048 if train else 7168) // d))
    return {"op": op, "train": train, "T": T, "d": d,
            "dtype": "bf16" if rng.random() < 0.7 else "fp32",
            "gate": rng.choice(["none", "all", "row"]), "post": rng.random() < 0.8,
            "pre": rng.random() < 0.8}


# ------------------------------------------------------------------------------ the inputs

ALPHA, BETA = 0.875, 0.7071     # scales of the residual stream and of the block's output


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 29)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    def weight4(rows, K, gs, zeros, *lead):
        """A 4-bit weight of rows of K values: codes, scales and zero points (None: 8)."""
        c = torch.randint(0, 256, (*lead, rows, K // 2), generator=g, device=DEV,
                          dtype=torch.uint8)
        s = torch.rand((*lead, rows, K // gs), generator=g, device=DEV) * 0.5 + 0.75
        s = (s * (K ** -0.5 / 4.6)).to(torch.bfloat16)
        z = torch.randint(5, 12, s.shape, generator=g, device=DEV, dtype=torch.uint8) \
            if zeros else None
        return c, s, z

    st = {"case": dict(case)}
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        # experts of unequal popularity, as a router in training has them
        st["logits"] = normal(T, E) + 0.5 * normal(1, E)
        st["bias"] = normal(E, scale=0.05) if case["bias"] else None
        if case["train"]:
            st["dw"] = normal(T, case["k"])
            st["dl_in"] = normal(T, E, scale=1e-2)        # the balance loss's share
    elif op == "w4":
        st["x"] = normal(case["M"], case["K"], dtype=torch.bfloat16)
        st["w"] = weight4(case["N"], case["K"], case["g"], case["zeros"])
    elif op == "moe":
        T, d, I, El, E, k = (case[n] for n in ("T", "d", "I", "El", "E", "k"))
        st["x"] = normal(T, d, dtype=torch.bfloat16)
        top = torch.topk(normal(T, E), k, dim=1)
        st["idx"] = top.indices.to(torch.int32).contiguous()
        st["tw"] = torch.softmax(top.values, dim=1).contiguous()
        for n, rows, K in (("gate", I, d), ("up", I, d), ("down", d, I)):
            st[n] = weight4(rows, K, case["g"], case["zeros"], El)
        st["y_in"] = normal(T, d, dtype=torch.bfloat16)   # the shared expert's output
    else:
        T, d, t = case["T"], case["d"], _TYPES[case["dtype"]]
        st["y"], st["res"] = normal(T, d, dtype=t, scale=0.5), normal(T, d, dtype=t, scale=2.0)
        st["w_post"] = (1.0 + normal(d, scale=0.1)).to(t) if case["post"] else None
        st["w_pre"] = (1.0 + normal(d, scale=0.1)).to(t) if case["pre"] else None
        st["gate"] = None
        if case["gate"] != "none":
            shape = (T, d) if case["gate"] == "row" else (d,)     # one value a token, or for all
            st["gate"] = torch.sigmoid(normal(*shape)).to(t)
        if case["train"]:
            st["dh"] = normal(T, d, dtype=t)
            st["dn"] = normal(T, d, dtype=t) if case["pre"] else None
    return st


# -------------------------------------------------------------- plain forms (float32 torch)

def _plain_route(st):
    c, l = st["case"], st["logits"]
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    l64 = l.double()
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l64))
    else:
        s = torch.exp(l64 - l64.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    pick = s if st["bias"] is None else s + st["bias"].double()
    low = torch.full((), -math.inf, dtype=torch.float64, device=DEV)
    if G > 1:
        left = pick.reshape(T, G, E // G)
        gs = torch.zeros(T, G, dtype=torch.float64, device=DEV)
        for _ in range(min(c["top"], E // G)):
            v, at = left.max(2, keepdim=True)
            gs = gs + v[:, :, 0]
            left = left.scatter(2, at, low.expand(T, G, 1))
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        for _ in range(c["Gk"]):
            at = gs.max(1, keepdim=True).indices
            keep.scatter_(1, at, True)
            gs = gs.scatter(1, at, low.expand(T, 1))
        pick = torch.where(keep[:, :, None], pick.reshape(T, G, E // G), low).reshape(T, E)
    idx = torch.empty(T, k, dtype=torch.int64, device=DEV)
    for j in range(k):
        at = pick.max(1, keepdim=True).indices
        idx[:, j:j + 1] = at
        pick = pick.scatter(1, at, low.expand(T, 1))
    p = torch.gather(s, 1, idx)
    w = c["scale"] * (p / p.sum(1, keepdim=True) if c["renorm"] else p)
    out = {"idx": idx.to(torch.int32), "w": w.float()}
    if c["train"]:
        dw, p = st["dw"], p.float()
        if c["renorm"]:
            tot = p.sum(1, keepdim=True)
            dp = c["scale"] / tot * (dw - (dw * p).sum(1, keepdim=True) / tot)
        else:
            dp = c["scale"] * dw
        if c["score"] == "sigmoid":
            dl = torch.zeros_like(l).scatter_(1, idx, dp * p * (1.0 - p))
        else:
            sf = s.float()
            ds = torch.zeros_like(l).scatter_(1, idx, dp)
            dl = sf * (ds - (ds * sf).sum(1, keepdim=True))
        out["dlogits"] = st["dl_in"] + dl
    return out


def _dequantise(c, s, z, g):
    """Float32 values of a 4-bit weight [..., K]: (code - zero) scale."""
    q = torch.stack([c & 15, c >> 4], -1).reshape(*s.shape, g).float()
    q = q - (8.0 if z is None else z.float()[..., None])
    return (q * s.float()[..., None]).reshape(*c.shape[:-1], -1)


def _plain_w4(st):
    c = st["case"]
    return (st["x"].float() @ _dequantise(*st["w"], c["g"]).T).to(_TYPES[c["out"]])


def _plain_moe(st):
    c = st["case"]
    T, k, El, e0 = c["T"], c["k"], c["El"], c["e0"]
    x, y = st["x"].float(), st["y_in"].float()
    idx = st["idx"].long() - e0
    tw = torch.where((idx >= 0) & (idx < El), st["tw"], 0.0)

    def matrix(n, e):         # transposed weights of the experts e (indices on the device)
        w, s, z = (None if t is None else t.index_select(0, e) for t in st[n])
        return _dequantise(w, s, z, c["g"]).transpose(1, 2)

    def ffn(a, e):            # a [len(e) or 1, rows, d]
        a = a.expand(e.shape[0], -1, -1)
        h, u = torch.bmm(a, matrix("gate", e)), torch.bmm(a, matrix("up", e))
        return torch.bmm(h / (1.0 + torch.exp(-h)) * u, matrix("down", e))

    n = max(1, 2 ** 27 // (c["d"] * c["I"]))              # experts whose weights are held at once
    if T * k <= El:           # few tokens: one FFN for each route
        e, rows = idx.reshape(-1).clamp(0, El - 1), x.repeat_interleave(k, 0)[:, None]
        p = torch.cat([ffn(rows[i:i + n], e[i:i + n]) for i in range(0, T * k, n)])
        y = y + (tw[:, :, None] * p.reshape(T, k, -1)).sum(1)
    else:                     # every local expert on all tokens, weighted
        every = torch.arange(El, device=DEV)
        for i in range(0, El, n):
            e = every[i:i + n]
            we = torch.where(idx[None] == e[:, None, None], tw[None], 0.0).sum(2)
            y = y + (we[:, :, None] * ffn(x[None], e)).sum(0)
    return y.to(torch.bfloat16)


def _plain_gnorm(st):
    c, t = st["case"], st["y"].dtype
    y = st["y"].float()
    wp = 1.0 if st["w_post"] is None else st["w_post"].float()
    gate = 1.0 if st["gate"] is None else st["gate"].float()
    ry = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) if c["post"] else 1.0
    v = y * ry
    u = v * wp
    h = (ALPHA * st["res"].float() + BETA * gate * u).to(t)
    out = {"h": h}
    hf = h.float()
    if c["pre"]:
        rh = torch.rsqrt((hf * hf).mean(1, keepdim=True) + EPS)
        nh = hf * rh
        out["n"] = (nh * st["w_pre"].float()).to(t)
    if not c["train"]:
        return out
    dh = st["dh"].float()
    if c["pre"]:
        dn = st["dn"].float()
        gn = dn * st["w_pre"].float()
        dh = dh + rh * (gn - nh * (gn * nh).mean(1, keepdim=True))
        out["dw_pre"] = (dn * nh).sum(0)
    out["dres"] = (ALPHA * dh).to(t)
    b = BETA * dh
    if st["gate"] is not None:
        dg = b * u
        out["dgate"] = dg.to(t) if c["gate"] == "row" else dg.sum(0)
    du = b * gate
    if c["post"]:
        out["dw_post"] = (du * v).sum(0)
        gv = du * wp
        du = ry * (gv - v * (gv * v).mean(1, keepdim=True))
    out["dy"] = du.to(t)
    return out


# ------------------------------------------------------- the library's calls (own is true)

def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _own_route(mok, st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    if "idx" not in st:       # outputs, kept from step to step by the program
        st["idx"], st["w"] = _empty(T, k, dtype=torch.int32), _empty(T, k)
        st["dl"] = _empty(T, E) if c["train"] else None
    mok.mok_topk_scored(st["logits"], k, st["idx"], st["w"], score=c["score"], bias=st["bias"],
                        n_groups=c["G"], topk_groups=c["Gk"], group_top=c["top"],
                        renorm=c["renorm"], scale=c["scale"])
    out = {"idx": st["idx"], "w": st["w"]}
    if c["train"]:
        mok.mok_topk_scored_backward(st["logits"], st["idx"], st["dw"], st["dl"],
                                     score=c["score"], renorm=c["renorm"], scale=c["scale"],
                                     dlogits_in=st["dl_in"])
        out["dlogits"] = st["dl"]
    return out


def _own_w4(mok, st):
    c = st["case"]
    if "out" not in st:
        st["out"] = _empty(c["M"], c["N"], dtype=_TYPES[c["out"]])
    codes, scales, zeros = st["w"]
    mok.mok_w4_gemm(st["x"], codes, scales, st["out"], zeros=zeros)
    return st["out"]


def _own_moe(mok, st):
    c = st["case"]
    if "layer" not in st:     # the handle of the weights, with its workspace
        st["layer"] = mok.MoeW4Layer(st["gate"], st["up"], st["down"], E=c["E"], k=c["k"],
                                     e0=c["e0"], max_tokens=c["T"])
        st["out"] = torch.empty_like(st["x"])
    st["layer"].forward(st["x"], st["idx"], st["tw"], st["out"], y_in=st["y_in"])
    return st["out"]


def _own_gnorm(mok, st):
    c, y = st["case"], st["y"]
    T, d = c["T"], c["d"]
    if "h" not in st:
        st["h"] = torch.empty_like(y)
        st["n"] = torch.empty_like(y) if c["pre"] else None
        if c["train"]:
            st["ry"] = _empty(T) if c["post"] else None
            st["rh"] = _empty(T) if c["pre"] else None
            st["dres"], st["dy"] = torch.empty_like(y), torch.empty_like(y)
            st["dgate"] = None
            if c["gate"] != "none":
                st["dgate"] = torch.empty_like(y) if c["gate"] == "row" else _empty(d)
            st["dw_post"] = _empty(d) if c["post"] else None
            st["dw_pre"] = _empty(d) if c["pre"] else None
            st["ws"] = _empty(mok.mok_gated_norm_backward_workspace_bytes(T, d),
                              dtype=torch.uint8)
    mok.mok_gated_norm(y, st["res"], EPS, st["h"], w_post=st["w_post"], gate=st["gate"],
                       w_pre=st["w_pre"], n=st["n"], rstd_y=st.get("ry"), rstd_h=st.get("rh"),
                       alpha=ALPHA, beta=BETA)
    out = {"h": st["h"]}
    if c["pre"]:
        out["n"] = st["n"]
    if not c["train"]:
        return out
    mok.mok_gated_norm_backward(st["dh"], y, st["dres"], st["dy"], st["ws"], dn=st["dn"],
                                h=st["h"], gate=st["gate"], w_post=st["w_post"],
                                w_pre=st["w_pre"], rstd_y=st["ry"], rstd_h=st["rh"],
                                dgate=st["dgate"], dw_post=st["dw_post"], dw_pre=st["dw_pre"],
                                alpha=ALPHA, beta=BETA)
    if c["pre"]:
        out["dw_pre"] = st["dw_pre"]
    out["dres"] = st["dres"]
    if st["gate"] is not None:
        out["dgate"] = st["dgate"]
    if c["post"]:
        out["dw_post"] = st["dw_post"]
    out["dy"] = st["dy"]
    return out


_PLAIN = {"route": _plain_route, "w4": _plain_w4, "moe": _plain_moe, "gnorm": _plain_gnorm}
_OWN = {"route": _own_route, "w4": _own_w4, "moe": _own_moe, "gnorm": _own_gnorm}


def run(state):
    op = state["case"]["op"]
    if own:
        import routing_grouped_expert_gemm_amd as mok
        return _OWN[op](mok, state)
    return _PLAIN[op](state)


# ------------------------------------------------------------------------- work of one pass

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # logits in, picks and weights out; training: dw and dlogits_in in, dlogits out
        n = 4 * T * E + 8 * T * k
        return {"bytes": n + (8 * T * E + 4 * T * k if case["train"] else 0),
                "flops": (10 if case["train"] else 6) * T * E}
    per = 0.5 + 2 / case["g"] + (1 / case["g"] if case["zeros"] else 0) \
        if op in ("w4", "moe") else 0
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        es = 2 if case["out"] == "bf16" else 4
        return {"bytes": int(2 * M * K + N * K * per + M * N * es), "flops": 2 * M * N * K}
    if op == "moe":
        T, d, I, E, El, k = (case[n] for n in ("T", "d", "I", "E", "El", "k"))
        # the weights of the local experts that some token picks (as many as even routing
        # touches); x, y_in, y; routing
        hit = El * (1.0 - (1.0 - k / E) ** T)
        return {"bytes": int(hit * 3 * d * I * per + 6 * T * d + 8 * T * k),
                "flops": int(6 * T * k * El / E * d * I)}
    T, d = case["T"], case["d"]
    es = 2 if case["dtype"] == "bf16" else 4
    # forward: y, residual in, h and n out; backward: dh, dn, y, h in, dres and dy out
    rows = 3 + case["pre"]
    if case["train"]:
        rows += 4 + 2 * case["pre"]
    if case["gate"] == "row":
        rows += 3 if case["train"] else 1
    return {"bytes": rows * T * d * es, "flops": (40 if case["train"] else 14) * T * d}


# -------------------------------------------------- the definitions once more, in float64

def _exact_choice(c, s, bias):
    """Experts of each row in the order of their scores, by sorting."""
    v = s.clone() if bias is None else torch.add(s, bias.to(torch.float64))
    T, E = v.shape
    if c["G"] > 1:
        size = E // c["G"]
        parts = v.view(T, c["G"], size)
        best = parts.sort(dim=2, descending=True).values[:, :, :c["top"]]
        worth = best[:, :, 0] if best.shape[2] == 1 else best[:, :, 0] + best[:, :, 1]
        order = worth.sort(dim=1, descending=True, stable=True).indices
        out = order[:, c["Gk"]:]                      # groups that are left out
        parts.scatter_(1, out[:, :, None].expand(-1, -1, size), -math.inf)
    return v.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]


def _exact_weight(c, w):
    codes, s, z = w
    q = torch.empty(*codes.shape, 2, dtype=torch.float64, device=DEV)
    q[..., 0] = torch.remainder(codes, 16)
    q[..., 1] = torch.div(codes, 16, rounding_mode="floor")
    q = q.flatten(-2).unflatten(-1, (-1, c["g"]))
    zero = torch.full(s.shape, 8.0, dtype=torch.float64, device=DEV) if z is None else z.double()
    return ((q - zero.unsqueeze(-1)) * s.double().unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64
    op, c = case["op"], case
    if op == "route":
        l = st["logits"].to(D)
        s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)
        idx = _exact_choice(c, s, st["bias"])
        with torch.enable_grad():
            lg = l.detach().requires_grad_(c["train"])
            sg = torch.sigmoid(lg) if c["score"] == "sigmoid" else torch.softmax(lg, dim=1)
            w = torch.take_along_dim(sg, idx, dim=1)
            if c["renorm"]:
                w = torch.div(w, w.sum(dim=1, keepdim=True))
            w = torch.mul(w, c["scale"])
            out = {"idx": idx.to(torch.int32), "w": w.detach()}
            if c["train"]:
                (grad,) = torch.autograd.grad(w, lg, grad_outputs=st["dw"].to(D))
                out["dlogits"] = torch.add(grad, st["dl_in"].to(D))
        return out
    if op == "w4":
        return torch.mm(st["x"].to(D), _exact_weight(c, st["w"]).t())
    if op == "moe":
        x, y = st["x"].to(D), st["y_in"].to(D)
        for e in range(c["El"]):
            t, j = torch.nonzero(st["idx"] == e + c["e0"], as_tuple=True)
            if t.numel() == 0:
                continue
            one = {n: _exact_weight(c, [None if v is None else v[e] for v in st[n]])
                   for n in ("gate", "up", "down")}
            a = x[t]
            h = torch.nn.functional.silu(torch.mm(a, one["gate"].t())) * torch.mm(a, one["up"].t())
            y.index_add_(0, t, torch.mm(h, one["down"].t()) * st["tw"][t, j].to(D)[:, None])
        return y
    t = st["y"].dtype
    y, res = st["y"].to(D), st["res"].to(D)

    def unit(v):
        return v / torch.sqrt(torch.linalg.vector_norm(v, dim=1) ** 2 / c["d"] + EPS)[:, None]

    wp = torch.ones(c["d"], dtype=D, device=DEV) if not c["post"] else st["w_post"].to(D)
    gate = torch.ones(c["d"], dtype=D, device=DEV) if st["gate"] is None else st["gate"].to(D)
    leaves = [v.detach().requires_grad_(c["train"]) for v in (y, res, wp, gate)]
    with torch.enable_grad():
        a = unit(leaves[0]) if c["post"] else leaves[0]
        hs = ALPHA * leaves[1] + BETA * leaves[3] * (a * leaves[2])
    h = hs.detach().to(t)                          # the residual stream as it is stored
    out = {"h": hs.detach()}
    if c["pre"]:
        hv = h.to(D).requires_grad_(c["train"])
        w2 = st["w_pre"].to(D).requires_grad_(c["train"])
        with torch.enable_grad():
            n = unit(hv) * w2
        out["n"] = n.detach()
    if not c["train"]:
        return out
    up = st["dh"].to(D)
    if c["pre"]:
        dh, out["dw_pre"] = torch.autograd.grad(n, (hv, w2), st["dn"].to(D))
        up = up + dh
    dy, out["dres"], dwp, dgate = torch.autograd.grad(hs, leaves, up)
    if st["gate"] is not None:
        out["dgate"] = dgate
    if c["post"]:
        out["dw_post"] = dwp
    out["dy"] = dy
    return out
