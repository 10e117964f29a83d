"""Measured calls of the decode-side operators: the router's expert choice
and its gradient, the experts' products with 4-bit weights, and the whole
expert layer for a few tokens.

`own = False` runs each operator in its plain form (elementary torch
operations, 32 bits or more); `own = True` makes the library's calls.

Sizes are those of a rank of a DeepSeek-V3-like layer (H = 7168, expert
width 2048, 256 or 384 experts, 8 per token, 8 ranks of 32 experts, 4096
tokens a rank) and small odd ones around them.
"""
import math

import torch

own = False

DEV = "cuda"
TINY = 1e-20  # added to a renormalised row's sum of scores

_LOGITS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the 4-bit float (sign bit 8)


def _cba():
    import combine_balancing_amd as cba
    return cba


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's expert choice in a decode step: latency only
        dict(name="route_token", op="route", T=1, E=256, K=8, dtype="fp32", scoring="sigmoid",
             bias=True, groups=8, top_groups=4, renorm=True, scale=2.5, masked=0.0),
        # a rank's 4096 tokens over 384 experts, softmax over bf16 logits
        # (many exact ties)
        dict(name="route_rank_bf16", op="route", T=4096, E=384, K=8, dtype="bf16",
             scoring="softmax", bias=False, groups=1, top_groups=1, renorm=True, scale=1.0,
             masked=0.0),
        # all ranks' tokens (the table the plan takes), bias and group limit
        dict(name="route_world", op="route", T=32768, E=256, K=8, dtype="fp32",
             scoring="sigmoid", bias=True, groups=8, top_groups=4, renorm=True, scale=2.5,
             masked=0.0),
        # the router's gradient over the same tokens in a training step
        dict(name="route_grad_world", op="route_grad", T=32768, E=256, K=8, dtype="fp32",
             scoring="sigmoid", renorm=True, scale=2.5, masked=0.0),
        # one dense product of one token (a gate/up projection's shape)
        dict(name="matvec_token", op="matvec", T=1, R=0, E=1, N=4096, K=7168, kind="int4",
             group=128, zeros=False, scales="bf16", per_route=False, out="bf16"),
        # down projections of 16 tokens' 8 routes, each with its own input row
        dict(name="matvec_routed_fp4", op="matvec", T=16, R=8, E=32, N=7168, K=2048, kind="fp4",
             group=32, zeros=False, scales="bf16", per_route=True, out="fp32"),
        # odd sizes: a last row tile and a last group that are cut short
        dict(name="matvec_odd", op="matvec", T=5, R=3, E=13, N=1001, K=2504, kind="int4",
             group=64, zeros=True, scales="fp16", per_route=False, out="bf16"),
        # one token through its 8 experts, bf16 weights
        dict(name="layer_token", op="layer", T=1, K=8, E=32, world=32, first=0, H=7168, I=2048,
             weights="bf16", group=0, zeros=False, scales="bf16", pruned=0.0, out="bf16"),
        # a decode batch on a rank that holds all 64 experts in 4 bits
        dict(name="layer_batch_int4", op="layer", T=32, K=8, E=64, world=64, first=0, H=7168,
             I=2048, weights="int4", group=128, zeros=False, scales="bf16", pruned=0.0,
             out="bf16"),
        # a rank's 32 of 256 experts for the world's 128 tokens: most routes
        # belong to other ranks, some are pruned
        dict(name="layer_rank", op="layer", T=128, K=8, E=32, world=256, first=64, H=7168,
             I=2048, weights="bf16", group=0, zeros=False, scales="bf16", pruned=0.1,
             out="bf16"),
        # small and odd: sizes of no multiple of a tile
        dict(name="layer_odd", op="layer", T=7, K=3, E=16, world=20, first=2, H=1000, I=344,
             weights="bf16", group=0, zeros=False, scales="bf16", pruned=0.0, out="fp32"),
        # 4-bit floats in groups of 32 for a mid-sized model's decode batch
        dict(name="layer_fp4", op="layer", T=9, K=4, E=64, world=64, first=0, H=2048, I=1408,
             weights="fp4", group=32, zeros=False, scales="fp16", pruned=0.0, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "matvec", "layer"])
    if op in ("route", "route_grad"):
        scoring = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        E = max(8, _log(rng, 8, 1000) // groups) * groups
        E = min(E, 1024 // groups * groups)
        top_groups = rng.randint(1, groups)
        # a renormalised single score is 1 whatever the logits: no gradient
        K = rng.randint(1 if op == "route" else 2, min(16, E // groups * top_groups))
        T = _log(rng, 1, 32768 * 256 // max(E, 256))
        c = dict(op=op, T=T, E=E, K=K, dtype=rng.choice(["fp32", "bf16", "fp16"]),
                 scoring=scoring, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                 masked=rng.choice([0.0, 0.0, 0.3]))
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, top_groups=top_groups)
        return c
    if op == "matvec":
        kind = rng.choice(["int4", "fp4"])
        R = rng.choice([0, 1, 2, 4, 8])
        N, K = _log(rng, 17, 8192), 8 * _log(rng, 4, 1024)
        E = 1 if R == 0 else max(2, min(_log(rng, 2, 64), 32 * 7168 * 2048 // (N * K)))
        return dict(op=op, T=_log(rng, 1, 128 if R < 4 else 64), R=R, E=E, N=N, K=K, kind=kind, group=rng.choice([32, 64, 128]),
                    zeros=kind == "int4" and rng.random() < 0.5,
                    scales=rng.choice(["bf16", "fp16"]),
                    per_route=R > 0 and rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]))
    weights = rng.choice(["bf16", "int4", "fp4"])
    E = _log(rng, 2, 28)
    world = E * rng.choice([1, 1, 2, 8])
    return dict(op=op, T=_log(rng, 1, 128), K=rng.randint(1, min(8, world)), E=E, world=world,
                first=0 if world == E else E * rng.randint(0, world // E - 1),
                H=8 * _log(rng, 16, 896), I=8 * _log(rng, 8, 256), weights=weights,
                group=0 if weights == "bf16" else rng.choice([32, 64, 128]),
                zeros=weights == "int4" and rng.random() < 0.5,
                scales=rng.choice(["bf16", "fp16"]), pruned=rng.choice([0.0, 0.1]),
                out=rng.choice(["bf16", "fp32"]))


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _logits(c, g):
    l = _randn(g, c["T"], c["E"]) + 0.5 * _randn(g, c["E"])  # some experts are popular
    if c["masked"]:
        off = torch.rand(c["T"], c["E"], generator=g, device=DEV) < c["masked"]
        off[::7] |= torch.arange(c["E"], device=DEV) >= 2  # rows with two experts left
        off[::21] = True                                   # and rows with none
        l = l.masked_fill(off, -math.inf)
    return l.to(_LOGITS[c["dtype"]])


def _routing(g, T, K, world):
    """Top-K ids of random logits (popular experts included) and scores."""
    l = _randn(g, T, world) + 0.5 * _randn(g, world)
    v, ids = torch.sort(l, dim=1, descending=True, stable=True)
    v, ids = v[:, :K], ids[:, :K]
    return ids.to(torch.int32).contiguous(), torch.softmax(v, dim=1).contiguous()


def _codes(c, g, E, N, K):
    """4-bit codes [E,N,K], scales [E,N,groups] and zero points, as a
    checkpoint holds them."""
    kind = c.get("kind") or c["weights"]
    G = -(-K // c["group"])
    codes = torch.randint(0, 16, (E, N, K), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(E, N, G, generator=g, device=DEV) + 0.5
    s = s / ((4.6 if kind == "int4" else 2.9) * math.sqrt(K))
    z = None
    if c["zeros"]:
        z = torch.randint(5, 12, (E, N, G), generator=g, device=DEV, dtype=torch.uint8)
    return dict(codes=codes, scales=s.to(_LOGITS[c["scales"]]), zeros=z, group=c["group"],
                kind=kind)


def _weights(c, g, E, N, K):
    if c.get("weights") == "bf16":
        return _randn(g, E, N, K, dtype=torch.bfloat16).mul_(1.0 / math.sqrt(K))
    w = _codes(c, g, E, N, K)
    if own:  # laid out once, when the weights are loaded
        return _cba().q4_pack(w["codes"], w["scales"], zeros=w["zeros"], group=w["group"],
                              kind=w["kind"])
    return w


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=c)
    if c["op"] in ("route", "route_grad"):
        st["logits"] = _logits(c, g)
        if c["op"] == "route":
            st["bias"] = 0.1 * _randn(g, c["E"]) if c["bias"] else None
        else:
            st["ids"], _ = _route_rows(st["logits"], c["K"], None, c["scoring"], 1, 1,
                                       c["renorm"], c["scale"])
            st["dscores"] = _randn(g, c["T"], c["K"])
        return st
    if c["op"] == "matvec":
        T, R = c["T"], c["R"]
        st["ids"] = _routing(g, T, min(R, c["E"]), c["E"])[0] if R else None
        if R > c["E"]:  # fewer experts than routes: the rest go nowhere
            st["ids"] = torch.cat([st["ids"], st["ids"].new_full((T, R - c["E"]), -1)], 1)
        shape = (T, R, c["K"]) if c["per_route"] else (T, c["K"])
        st["x"] = _randn(g, *shape, dtype=torch.bfloat16)
        st["w"] = _weights(c, g, c["E"], c["N"], c["K"])
        st["out"] = torch.zeros((T, R, c["N"]) if R else (T, c["N"]), device=DEV,
                                dtype=_LOGITS[c["out"]])
        return st
    T, K = c["T"], c["K"]
    st["ids"], st["scores"] = _routing(g, T, K, c["world"])
    st["mask"] = None
    if c["pruned"]:
        st["mask"] = (torch.rand(T, K, generator=g, device=DEV) >= c["pruned"]).to(torch.uint8)
    st["x"] = _randn(g, T, c["H"], dtype=torch.bfloat16)
    st["w13"] = _weights(c, g, c["E"], 2 * c["I"], c["H"])
    st["w2"] = _weights(c, g, c["E"], c["H"], c["I"])
    st["out"] = torch.zeros(T, c["H"], device=DEV, dtype=_LOGITS[c["out"]])
    if own:
        st["workspace"] = _cba().moe_layer_workspace(T, K, c["I"])
    return st


# ------------------------------------------------------------ plain forms

def _live_scores(logits, scoring):
    """Scores of all experts in 64 bits; an expert at -inf has none."""
    l = logits.double()
    live = l > -math.inf
    if scoring == "softmax":
        top = l.amax(1, keepdim=True)
        e = torch.where(live, torch.exp(l - torch.where(top > -math.inf, top, 0.0)), 0.0)
        p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        p = torch.where(live, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    return l, live, p


def _route_rows(logits, K, bias, scoring, groups, top_groups, renorm, scale):
    # in 64 bits: a choice next to a border must not hang on rounding
    T, E = logits.shape
    l, live, p = _live_scores(logits, scoring)
    c = torch.where(live, l if bias is None else p + bias.double(), -math.inf)
    if groups > 1:
        per = torch.sort(c.view(T, groups, E // groups), dim=2, descending=True)[0]
        best = per[:, :, 0]
        if bias is not None and E // groups > 1:
            second = per[:, :, 1]
            best = best + torch.where(second > -math.inf, second, 0.0)
        order = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :top_groups]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=logits.device)
        keep.scatter_(1, order, True)
        c = torch.where(keep.repeat_interleave(E // groups, 1), c, -math.inf)
    v, ids = torch.sort(c, dim=1, descending=True, stable=True)
    v, ids = v[:, :K], ids[:, :K]
    w = torch.where(v > -math.inf, p.gather(1, ids), 0.0)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + TINY)
    ids = torch.where(v > -math.inf, ids, -1)
    return ids.to(torch.int32), (w * scale).float()


def _route_grad_rows(logits, ids, dscores, scoring, renorm, scale):
    l, live, p = _live_scores(logits, scoring)
    ok = ids >= 0
    at = ids.clamp_min(0).long()
    s = torch.where(ok, p.gather(1, at), 0.0)
    g = torch.where(ok, dscores.double() * scale, 0.0)
    if renorm:
        d = s.sum(1, keepdim=True) + TINY
        g = (g - (g * (s / d)).sum(1, keepdim=True)) / d
        g = torch.where(ok, g, 0.0)
    dp = torch.zeros_like(p).scatter_add_(1, at, g)
    if scoring == "softmax":
        dl = p * (dp - (dp * p).sum(1, keepdim=True))
    else:
        dl = dp * p * (1.0 - p)
    return dl.to(logits.dtype)


def _dense(w, e, dtype=torch.float32):
    """Matrix e of a weight set, [N, K] in `dtype`."""
    if isinstance(w, torch.Tensor):
        return w[e].to(dtype)
    codes, K = w["codes"][e], w["codes"].shape[2]
    if w["kind"] == "int4":
        v = codes.to(dtype)
        z = 8.0 if w["zeros"] is None else (
            w["zeros"][e].to(dtype).repeat_interleave(w["group"], 1)[:, :K])
        v = v - z
    else:
        t = torch.tensor(_FP4 + tuple(-m for m in _FP4), dtype=dtype, device=codes.device)
        v = t[codes.int()]
    return v * w["scales"][e].to(dtype).repeat_interleave(w["group"], 1)[:, :K]


def _matvec_rows(x, w, ids, out, dtype=torch.float32):
    T = x.shape[0]
    if ids is None:
        y = x.to(dtype) @ _dense(w, 0, dtype).t()
        return y.to(out) if out is not None else y
    R = ids.shape[1]
    xr = (x if x.dim() == 3 else x[:, None].expand(T, R, x.shape[1])).reshape(T * R, -1).to(dtype)
    flat = ids.reshape(-1, 1)
    y = None
    for e in range(w["codes"].shape[0]):
        ye = xr @ _dense(w, e, dtype).t()
        y = torch.zeros_like(ye) if y is None else y
        y = torch.where(flat == e, ye, y)
    y = y.view(T, R, -1)
    return y.to(out) if out is not None else y


def _layer_rows(st, dtype=torch.float32):
    c, x = st["case"], st["x"].to(dtype)
    score = st["scores"].to(dtype)
    if st["mask"] is not None:
        score = torch.where(st["mask"] != 0, score, 0.0)
    y = torch.zeros(x.shape, dtype=dtype, device=x.device)
    for e in range(c["E"]):
        mine = st["ids"] == c["first"] + e
        if st["mask"] is not None:
            mine = mine & (st["mask"] != 0)
        gu = x @ _dense(st["w13"], e, dtype).t()
        gate, up = gu[:, :c["I"]], gu[:, c["I"]:]
        h = gate / (1.0 + torch.exp(-gate)) * up
        ye = h @ _dense(st["w2"], e, dtype).t()
        y = y + torch.where(mine, score, 0.0).sum(1, keepdim=True) * ye
    return y


# -------------------------------------------------------------------- run

def run(st):
    c = st["case"]
    if c["op"] == "route":
        if own:
            return _cba().route(st["logits"], c["K"], bias=st["bias"], scoring=c["scoring"],
                                n_group=c["groups"], topk_group=c["top_groups"],
                                renormalize=c["renorm"], scale=c["scale"])
        return _route_rows(st["logits"], c["K"], st["bias"], c["scoring"], c["groups"],
                           c["top_groups"], c["renorm"], c["scale"])
    if c["op"] == "route_grad":
        if own:
            return _cba().route_grad(st["logits"], st["ids"], st["dscores"],
                                     scoring=c["scoring"], renormalize=c["renorm"],
                                     scale=c["scale"])
        return _route_grad_rows(st["logits"], st["ids"], st["dscores"], c["scoring"],
                                c["renorm"], c["scale"])
    if c["op"] == "matvec":
        if own:
            return _cba().expert_matvec_q4(st["x"], st["w"], ids=st["ids"], out=st["out"])
        return _matvec_rows(st["x"], st["w"], st["ids"], st["out"].dtype)
    if own:
        ob, of = (st["out"], None) if c["out"] == "bf16" else (None, st["out"])
        ob, of = _cba().moe_layer(st["x"], st["ids"], st["scores"], st["w13"], st["w2"],
                                  first=c["first"], mask=st["mask"], out_bf16=ob, out_f32=of,
                                  workspace=st["workspace"])
        return ob if c["out"] == "bf16" else of
    return _layer_rows(st).to(st["out"].dtype)


# ------------------------------------------------------------------- work

def _weight_bytes(c, E, N, K):
    if c.get("weights") == "bf16":
        return 2 * E * N * K
    G = -(-K // c["group"])
    return E * N * (K / 2 + G * (3 if c["zeros"] else 2))


def _reached(T, K, world, E):
    """Expected number of E of `world` equally likely experts that T tokens
    with K distinct choices each reach."""
    return E * (1.0 - (1.0 - min(K, world) / world) ** T)


def work(case):
    c = case
    if c["op"] in ("route", "route_grad"):
        T, E, K = c["T"], c["E"], c["K"]
        lb = 4 if c["dtype"] == "fp32" else 2
        if c["op"] == "route":
            return {"bytes": T * E * lb + T * K * 8 + (4 * E if c["bias"] else 0),
                    "flops": 4.0 * T * E}
        return {"bytes": 2 * T * E * lb + T * K * 8, "flops": 4.0 * T * E}
    osz = 2 if c["out"] == "bf16" else 4
    if c["op"] == "matvec":
        routes = c["T"] * max(1, min(c["R"], c["E"]))
        E = _reached(c["T"], c["R"], c["E"], c["E"]) if c["R"] else 1
        rows = c["T"] * (c["R"] if c["per_route"] else 1)
        return {"bytes": _weight_bytes(c, E, c["N"], c["K"]) + rows * c["K"] * 2
                + routes * c["N"] * osz, "flops": 2.0 * routes * c["N"] * c["K"]}
    T, K, H, I = c["T"], c["K"], c["H"], c["I"]
    E = _reached(T, K * (1.0 - c["pruned"]), c["world"], c["E"])
    routes = T * K * (1.0 - c["pruned"]) * c["E"] / c["world"]
    return {"bytes": _weight_bytes(c, E, 2 * I, H) + _weight_bytes(c, E, H, I)
            + T * H * (2 + osz) + T * K * 8, "flops": 6.0 * routes * H * I}


# ------------------------------------------------------------------ exact

def _exact_values(w, e):
    """Matrix e in 64 bits, group by group."""
    if isinstance(w, torch.Tensor):
        return w[e].double()
    codes, g = w["codes"][e], w["group"]
    out = torch.empty(codes.shape, dtype=torch.float64, device=codes.device)
    for i in range(w["scales"].shape[2]):
        q = codes[:, i * g:(i + 1) * g].long()
        if w["kind"] == "int4":
            v = (q - (8 if w["zeros"] is None else w["zeros"][e][:, i:i + 1].long())).double()
        else:  # sign, two exponent bits, one mantissa bit; exponent 0 is subnormal
            m, x = (q & 1).double(), (q >> 1 & 3)
            v = torch.where(x == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((x - 1).double()))
            v = torch.where(q >= 8, -v, v)
        out[:, i * g:(i + 1) * g] = v * w["scales"][e][:, i:i + 1].double()
    return out


def _exact_route(st):
    """Repeatedly takes the best remaining expert."""
    c = st["case"]
    l = st["logits"].double()
    T, E = l.shape
    live = ~torch.isinf(l)
    row_live = live.any(1, keepdim=True)
    if c["scoring"] == "softmax":
        p = torch.softmax(torch.where(row_live, l, 0.0), 1) * live
    else:
        p = torch.sigmoid(l)
    val = l if st["bias"] is None else p + st["bias"].double()
    val = val.masked_fill(~live, -math.inf)
    idx = torch.arange(E, device=l.device)

    def take(v):  # the first index of the largest value, and whether one is left
        top = v.amax(1, keepdim=True)
        n = v.shape[1]
        at = torch.where(v == top, idx[:n], n).amin(1, keepdim=True)
        return at, top

    if c["groups"] > 1:
        per = E // c["groups"]
        gs = []
        for i in range(c["groups"]):
            v = val[:, i * per:(i + 1) * per]
            at, a = take(v)
            if st["bias"] is not None:
                b = v.scatter(1, at, -math.inf).amax(1, keepdim=True)
                a = a + torch.where(torch.isinf(b), 0.0, b)
            gs.append(a)
        gs = torch.cat(gs, 1)
        keep = torch.zeros_like(gs, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            at, top = take(gs)
            keep.scatter_(1, at, True)
            gs = gs.scatter(1, at, -math.inf)
        val = torch.where(keep[:, idx // per], val, -math.inf)
    ids, w = [], []
    for _ in range(c["K"]):
        at, top = take(val)
        ok = ~torch.isinf(top)
        ids.append(torch.where(ok, at, -1))
        w.append(torch.where(ok, p.gather(1, at), 0.0))
        val = val.scatter(1, at, -math.inf)
    ids, w = torch.cat(ids, 1), torch.cat(w, 1)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + TINY)
    return ids, w * c["scale"]


def _exact_route_grad(st):
    """Autograd in 64 bits through the scores of the chosen experts."""
    c = st["case"]
    l = st["logits"].double()
    live = ~torch.isinf(l)
    l = torch.where(live, l, 0.0).requires_grad_(True)
    if c["scoring"] == "softmax":
        e = torch.exp(l - l.detach().amax(1, keepdim=True)) * live
        p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        p = torch.sigmoid(l) * live
    ok = st["ids"] >= 0
    s = p.gather(1, st["ids"].clamp_min(0).long()) * ok
    if c["renorm"]:
        s = s / (s.sum(1, keepdim=True) + TINY)
    (s * c["scale"] * st["dscores"].double()).sum().backward()
    return l.grad


def _exact_matvec(st):
    x, w, ids = st["x"].double(), st["w"], st["ids"]
    if ids is None:
        return x @ _exact_values(w, 0).t()
    T, R = ids.shape
    y = torch.zeros(T * R, w["codes"].shape[1], dtype=torch.float64, device=x.device)
    flat = ids.reshape(-1)
    for e in flat.unique().tolist():
        if e < 0:
            continue
        rows = (flat == e).nonzero()[:, 0]
        xe = x.reshape(T * R, -1)[rows] if x.dim() == 3 else x[rows // R]
        y[rows] = xe @ _exact_values(w, e).t()
    return y.view(T, R, -1)


def _exact_layer(st):
    c, x = st["case"], st["x"].double()
    y = torch.zeros_like(x)
    keep = torch.ones_like(st["ids"], dtype=torch.bool) if st["mask"] is None else st["mask"] > 0
    for e in range(c["E"]):
        t, k = ((st["ids"] == c["first"] + e) & keep).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        w = _exact_values(st["w13"], e)
        gate, up = x[t] @ w[:c["I"]].t(), x[t] @ w[c["I"]:].t()
        h = gate * torch.sigmoid(gate) * up
        y.index_add_(0, t, st["scores"][t, k].double()[:, None]
                     * (h @ _exact_values(st["w2"], e).t()))
    return y


def exact(case, seed):
    global own
    was, own = own, False  # the inputs as a checkpoint holds them, not laid out
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "route":
        return _exact_route(st)
    if case["op"] == "route_grad":
        return _exact_route_grad(st)
    if case["op"] == "matvec":
        return _exact_matvec(st)
    return _exact_layer(st)
