"""Cases for what stands in front of the MoE exchange:

  norm, norm_bwd          the root-mean-square norm with the residual's addition,
                          results in the rows' type or as rows of 8 bits, and its
                          gradients
  route, route_bwd        the router: scores, a bias for balance, groups, the K best
                          experts and their weights, what each expert gets, and the
                          gradient of the logits
  quantize, dequantize    rows to 8 bits (e4m3 with a power of two for each 32
                          values) and back
  experts_q8              the experts' matrix products on such rows, ragged by expert

With ``own`` false, ``run`` computes an operator in elementary torch
operations; with ``own`` true it calls the library.

A row of 8 bits: H values of e4m3, zeros up to a multiple of 128; one byte for
each 32 of them, the exponent e + 127 of their scale 2^e, the smallest one (of
byte 0 at least) with largest magnitude <= 448 * 2^e; the row ends at a multiple
of 128 bytes.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # Serving: one token's hidden state joins the residual stream and goes
        # to its experts in 8 bits; latency.
        dict(name="norm_token_q8", op="norm", dtype="bf16", R=1, T=1, H=2048, add=True, out="q8"),
        # Training at the expert-parallel dispatch workload's size: 8 ranks x 4096
        # tokens, hidden 2048, residual added, rows for the router and the experts.
        dict(name="norm_train_bf16", op="norm", dtype="bf16", R=8, T=4096, H=2048, add=True, out="y"),
        # The same rows in 8 bits, as an 8-bit dispatch sends them.
        dict(name="norm_train_q8", op="norm", dtype="bf16", R=8, T=4096, H=2048, add=True, out="q8"),
        # The training layer's gradients, with the residual stream's own.
        dict(name="norm_bwd_train_bf16", op="norm_bwd", dtype="bf16", R=8, T=4096, H=2048, add=True),
        # A small fp32 layer with odd sizes.
        dict(name="norm_bwd_odd_f32", op="norm_bwd", dtype="f32", R=2, T=701, H=1036, add=False),
        # A router of many experts: sigmoid scores, a bias for balance, 4 of 8
        # groups by their two best, renormalised and scaled weights, counts and
        # sums of the scores.
        dict(name="route_groups", op="route", R=8, T=4096, E=256, K=8, score="sigmoid", bias=True,
             groups=8, kept=4, group_top=2, renorm=True, scale=2.5, stats=True),
        # Serving: one token's choice of 6 of 64 experts.
        dict(name="route_token", op="route", R=1, T=1, E=64, K=6, score="softmax", bias=False,
             groups=1, kept=1, group_top=1, renorm=True, scale=1.0, stats=False),
        # The gradient of the dispatch workload's router, balance loss included.
        dict(name="route_bwd_train", op="route_bwd", R=8, T=4096, E=64, K=6, score="softmax", bias=False,
             groups=1, kept=1, group_top=1, renorm=True, scale=1.0, stats=True),
        # A rank's expert weights laid out in 8 bits.
        dict(name="quantize_weights", op="quantize", dtype="bf16", R=2, rows=8 * 1408, H=2048),
        # Rows that arrived in 8 bits, as the weight gradient reads them.
        dict(name="dequantize_rows", op="dequantize", dtype="bf16", R=2, rows=24571, H=2048),
        # The products of the dispatch workload's layer on 8-bit rows.
        dict(name="experts_q8_train", op="experts_q8", R=8, T=4096, E=64, K=6, H=2048, F=1024, skew=0.5,
             route=11),
        # Serving: a decode batch of 48 tokens over all 64 experts, few rows each.
        dict(name="experts_q8_batch", op="experts_q8", R=1, T=48, E=64, K=6, H=2048, F=1024, skew=0.5,
             route=16),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "route", "route", "route_bwd", "quantize", "dequantize",
                     "experts_q8", "experts_q8"])
    R = rng.choice([1, 1, 2, 4, 8])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        H = 8 * _log(rng, 4, 2048)
        T = max(1, min(_log(rng, 1, 16384), int(120e6 / (R * H * SIZE[dt]))))
        case = dict(op=op, dtype=dt, R=R, T=T, H=H, add=rng.random() < 0.6)
        if op == "norm":
            case["out"] = rng.choice(["y", "q8", "both"])
        return case
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        E = groups * rng.choice([3, 4, 8, 16, 32, 60])
        kept = rng.randint(1, groups)
        K = rng.randint(1, min(8, kept * (E // groups)))
        T = max(1, min(_log(rng, 1, 16384), int(8e6 / (R * E))))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, R=R, T=T, E=E, K=K, score=score, bias=rng.random() < 0.5, groups=groups,
                    kept=kept, group_top=rng.choice([1, 2]),
                    renorm=K > 1 and rng.random() < 0.7,  # one renormalised weight is a constant
                    scale=rng.choice([1.0, 2.5]), stats=rng.random() < 0.5)
    if op in ("quantize", "dequantize"):
        H = 8 * _log(rng, 4, 2048)
        rows = max(1, min(_log(rng, 1, 65536), int(120e6 / (R * H * SIZE[dt]))))
        return dict(op=op, dtype=dt, R=R, rows=rows, H=H)
    E = R * rng.choice([1, 2, 3, 4, 8])
    K = rng.randint(1, min(E, 8))
    H, F = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 512)
    # at most a third of the largest listed case's flops
    T = max(1, min(_log(rng, 1, 8192), int(0.27e12 / (2.0 * R * K * H * F))))
    return dict(op=op, R=R, T=T, E=E, K=K, H=H, F=F, skew=rng.choice([0.0, 0.5, 1.5]),
                route=rng.randrange(1 << 30))


# ------------------------------------------------------------------ shapes
def expert_counts(case):
    """[R x E] rows each rank sends to each expert: T*K rows a rank, spread over
    the experts by a popularity that `skew` makes uneven."""
    rng = np.random.default_rng(case["route"])
    p = np.exp(case["skew"] * rng.normal(size=case["E"]))
    if case["skew"] >= 1.0:
        p[rng.random(case["E"]) < 0.2] = 0.0  # experts without a row
        p[rng.integers(case["E"])] += 1.0
    return rng.multinomial(case["T"] * case["K"], p / p.sum(), size=case["R"]).astype(np.int64)


def expert_rows(case):
    """Per rank d, the rows of each of its experts: [R][E/R]."""
    return expert_counts(case).sum(axis=0).reshape(case["R"], case["E"] // case["R"])


def row_bytes(H):
    blocks = -(-H // 128)
    return 128 * (blocks + -(-4 * blocks // 128))


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, s = case["R"] * case["T"], SIZE[case["dtype"]]
        row, small = case["H"] * s, n * 4 + case["R"] * case["H"] * s
        if op == "norm":
            moved = (3 if case["add"] else 1) * row
            moved += row if case["out"] != "q8" else 0
            moved += case["H"] * 33 / 32 if case["out"] != "y" else 0
            return {"bytes": n * moved + small, "flops": 5 * n * case["H"]}
        return {"bytes": n * (4 if case["add"] else 3) * row + small + case["R"] * case["H"] * 4,
                "flops": 10 * n * case["H"]}
    if op in ("route", "route_bwd"):
        n, E, K = case["R"] * case["T"], case["E"], case["K"]
        if op == "route":
            return {"bytes": n * (E * 4 + K * 8) + (case["R"] * E * 12 if case["stats"] else 0),
                    "flops": 10 * n * E}
        return {"bytes": n * (E * 8 + K * 8) + (case["R"] * E * 4 if case["stats"] else 0),
                "flops": 10 * n * E}
    if op in ("quantize", "dequantize"):
        n, H = case["R"] * case["rows"], case["H"]
        return {"bytes": n * (H * SIZE[case["dtype"]] + H * 33 / 32), "flops": 3 * n * H}
    rows = expert_rows(case)
    n, used = int(rows.sum()), int((rows > 0).sum())
    H, F = case["H"], case["F"]
    return {"bytes": n * (H * 33 / 32 + F * 2) + used * H * F * 33 / 32,
            "flops": 2 * n * H * F}


# ------------------------------------------------------------------ inputs
def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale


def _pack(x):
    """Rows of 8 bits of x [..., H], as bytes."""
    H = x.shape[-1]
    blocks = -(-H // 128)
    v = torch.zeros(*x.shape[:-1], blocks * 128, device="cuda")
    v[..., :H] = x.float()
    v = v.view(*x.shape[:-1], blocks * 4, 32)
    e = _exponent(v)
    rows = torch.zeros(*x.shape[:-1], row_bytes(H), dtype=torch.uint8, device="cuda")
    rows[..., :blocks * 128] = torch.ldexp(v, -e).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    rows[..., blocks * 128:blocks * 132] = (e.squeeze(-1) + 127).to(torch.uint8)
    return rows


def _ranks(rows, per_rank):
    """One tensor per rank of the rows of all of them."""
    return list(rows.split(per_rank))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, R = case["op"], case["R"]
    st = {"case": case}
    if op in ("norm", "norm_bwd"):
        dt, T, H = DT[case["dtype"]], case["T"], case["H"]
        channels = torch.exp(0.5 * _normal(g, (H,)))  # some are larger than others
        st["w"] = (1 + 0.1 * _normal(g, (H,))).to(dt)
        if op == "norm":
            st["x"] = _normal(g, (R, T, H)).to(dt)
            if case["add"]:
                st["res"] = (_normal(g, (R, T, H), 2.0) * channels).to(dt)
                st["h"] = torch.empty(R, T, H, dtype=dt, device="cuda")
            if case["out"] != "q8":
                st["y"] = torch.empty(R, T, H, dtype=dt, device="cuda")
            if case["out"] != "y":
                st["q"] = torch.empty(R, T, row_bytes(H), dtype=torch.uint8, device="cuda")
                st["values"] = torch.empty(R, T, H, dtype=torch.bfloat16, device="cuda")
            st["rstd"] = torch.empty(R, T, dtype=torch.float32, device="cuda")
        else:
            st["h"] = (_normal(g, (R, T, H), 2.0) * channels).to(dt)
            st["dy"] = _normal(g, (R, T, H), 0.02).to(dt)
            st["rstd"] = torch.rsqrt(st["h"].double().square().mean(dim=-1) + EPS).float()
            if case["add"]:
                st["dh"] = _normal(g, (R, T, H), 0.02).to(dt)
            st["dx"] = torch.empty(R, T, H, dtype=dt, device="cuda")
            st["dw"] = torch.empty(R, H, dtype=torch.float32, device="cuda")
    elif op in ("route", "route_bwd"):
        T, E, K = case["T"], case["E"], case["K"]
        st["logits"] = _normal(g, (R, T, E), 1.5)
        st["bias"] = _normal(g, (E,), 0.05) if case["bias"] else None
        if op == "route":
            st["topk"] = torch.empty(R, T, K, dtype=torch.int32, device="cuda")
            st["weights"] = torch.empty(R, T, K, dtype=torch.float32, device="cuda")
            if case["stats"]:
                st["counts"] = torch.empty(R, E, dtype=torch.int64, device="cuda")
                st["sums"] = torch.empty(R, E, dtype=torch.float32, device="cuda")
        else:
            st["topk"] = _choose(case, st["logits"], st["bias"])[0].to(torch.int32)
            st["dweights"] = _normal(g, (R, T, K), 0.1)
            if case["stats"]:
                st["dsums"] = _normal(g, (R, E), 0.01)
            st["dlogits"] = torch.empty(R, T, E, dtype=torch.float32, device="cuda")
    elif op in ("quantize", "dequantize"):
        dt, n, H = DT[case["dtype"]], case["rows"], case["H"]
        x = _normal(g, (R, n, H), 1 / math.sqrt(H) if op == "quantize" else 1.0).to(dt)
        if op == "quantize":
            st["x"], st["q"] = x, torch.empty(R, n, row_bytes(H), dtype=torch.uint8, device="cuda")
        else:
            st["q"] = _pack(x)
        st["values"] = torch.empty(R, n, H, dtype=dt, device="cuda")
    else:
        E, H, F = case["E"], case["H"], case["F"]
        rows = expert_rows(case)
        st["ecnt"], st["rows"] = expert_counts(case), rows.reshape(-1).tolist()
        per_rank = rows.sum(axis=1).tolist()
        total = sum(per_rank)
        st["exp"] = _pack(_normal(g, (total, H)))
        st["w"] = _pack(_normal(g, (E, F, H), 1 / math.sqrt(H)))
        st["out"] = torch.empty(total, F, dtype=torch.bfloat16, device="cuda")
        st["per_rank"] = per_rank
    if own:
        import collective_communication_reduce_amd as ccr
        st["ctx"] = ccr.Context(torch.cuda.current_device())
        if op == "norm_bwd":
            st["work"] = torch.empty(ccr.ccr_rms_norm_work(R, case["T"], case["H"]), device="cuda")
        if op == "route" and case["stats"]:
            st["work"] = torch.empty(ccr.ccr_moe_route_work(R, case["T"], case["E"]), device="cuda")
    return st


# ------------------------------------------------------------- plain forms
def _exponent(v):
    """The exponent of each block's scale, [..., 1] of [..., 32]."""
    m, e = torch.frexp(v.abs().amax(dim=-1, keepdim=True))  # m in [1/2, 1); 448 = 7/8 * 2^9
    return torch.where(m == 0, -127, torch.clamp(torch.where(m <= 0.875, e - 9, e - 8), min=-127))


def _q8_values(y):
    """What rows of 8 bits of y [..., H] stand for."""
    H = y.shape[-1]
    v = torch.nn.functional.pad(y, (0, -H % 32)).unflatten(-1, (-1, 32))
    e = _exponent(v)
    q = torch.ldexp(v, -e).to(torch.float8_e4m3fn).to(y.dtype)
    return torch.ldexp(q, e).flatten(-2)[..., :H]


def _unpack(rows, H):
    """The values of packed rows, in fp32."""
    blocks = -(-H // 128)
    q = rows[..., :blocks * 128].view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    e = rows[..., blocks * 128:blocks * 132].int() - 127
    return torch.ldexp(q, e.unsqueeze(-1)).flatten(-2)[..., :H]


def _scores(case, logits):
    l = logits.double()
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    z = torch.exp(l - l.max(dim=-1, keepdim=True).values)
    return z / z.sum(dim=-1, keepdim=True)


def _choose(case, logits, bias):
    """(experts chosen, scores of all): in 64 bits, since two experts may lie next
    to each other at the border.  Without a bias the logits order the experts."""
    s = _scores(case, logits)
    key = logits.double() if bias is None else s + bias.double()
    if case["kept"] < case["groups"]:
        by = key if case["group_top"] == 1 else (s if bias is None else key)
        by = by.unflatten(-1, (case["groups"], -1)).sort(dim=-1, descending=True).values
        value = by[..., :case["group_top"]].sum(dim=-1)
        best = value.sort(dim=-1, descending=True, stable=True).indices[..., :case["kept"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter(-1, best, True)
        keep = keep.repeat_interleave(case["E"] // case["groups"], dim=-1)
        key = torch.where(keep, key, float("-inf"))
    return key.sort(dim=-1, descending=True, stable=True).indices[..., :case["K"]], s


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        dt, res = DT[case["dtype"]], {}
        h = st["x"]
        if case["add"]:
            h = res["h"] = (st["x"].float() + st["res"].float()).to(dt)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(dim=-1) + EPS)
        y = hf * rstd[..., None] * st["w"].float()
        if case["out"] != "q8":
            res["y"] = y.to(dt)
        if case["out"] != "y":
            res["values"] = _q8_values(y).to(torch.bfloat16)  # holds every value of 8 bits
        return {**res, "rstd": rstd}
    if op == "norm_bwd":
        hh = st["h"].float() * st["rstd"][..., None]
        dy = st["dy"].float()
        g = dy * st["w"].float()
        dx = st["rstd"][..., None] * (g - hh * (g * hh).mean(dim=-1, keepdim=True))
        if case["add"]:
            dx = dx + st["dh"].float()
        return {"dx": dx.to(st["dx"].dtype), "dw": (dy * hh).sum(dim=1)}
    if op == "route":
        topk, s = _choose(case, st["logits"], st["bias"])
        w = s.gather(-1, topk)
        if case["renorm"]:
            w = w / w.sum(dim=-1, keepdim=True)
        res = {"topk": topk.to(torch.int32), "weights": (w * case["scale"]).float()}
        if case["stats"]:
            at = topk.flatten(1)
            res["counts"] = torch.zeros(case["R"], case["E"], dtype=torch.int64, device="cuda").scatter_add(
                1, at, torch.ones_like(at))
            res["sums"] = s.sum(dim=1).float()
        return res
    if op == "route_bwd":
        l, at = st["logits"], st["topk"].long()
        if case["score"] == "sigmoid":
            s = 1 / (1 + torch.exp(-l))
        else:
            z = torch.exp(l - l.max(dim=-1, keepdim=True).values)
            s = z / z.sum(dim=-1, keepdim=True)
        dw = st["dweights"] * case["scale"]
        if case["renorm"]:
            c = s.gather(-1, at)
            total = c.sum(dim=-1, keepdim=True)
            dw = (dw - (dw * c).sum(dim=-1, keepdim=True) / total) / total
        ds = torch.zeros_like(l).scatter_add(-1, at, dw)
        if case["stats"]:
            ds = ds + st["dsums"][:, None, :]
        if case["score"] == "sigmoid":
            return s * (1 - s) * ds
        return s * (ds - (s * ds).sum(dim=-1, keepdim=True))
    if op == "quantize":
        return _q8_values(st["x"].float()).to(DT[case["dtype"]])
    if op == "dequantize":
        return _unpack(st["q"], case["H"]).to(DT[case["dtype"]])
    exp, w = _unpack(st["exp"], case["H"]).split(st["rows"]), _unpack(st["w"], case["H"])
    return torch.cat([x @ w[e].t() for e, x in enumerate(exp)]).to(torch.bfloat16)


def run(state):
    if not own:
        return _plain(state)
    import collective_communication_reduce_amd as ccr
    st, case, op, ctx, R = state, state["case"], state["case"]["op"], state["ctx"], state["case"]["R"]
    if op == "norm":
        more, res = {}, {}
        if case["add"]:
            more.update(residual=st["res"].unbind(), h=st["h"].unbind())
            res["h"] = st["h"]
        if case["out"] != "q8":
            more["y"], res["y"] = st["y"].unbind(), st["y"]
        if case["out"] != "y":
            more["q"], res["values"] = st["q"].unbind(), st["values"]
        ccr.ccr_rms_norm(ctx, st["x"].unbind(), [st["w"]] * R, rstd=st["rstd"].unbind(), eps=EPS, **more)
        if case["out"] != "y":  # 8 bits are given back as the values they stand for
            ccr.ccr_dequantize_rows(ctx, st["q"].unbind(), st["values"].unbind())
        return {**res, "rstd": st["rstd"]}
    if op == "norm_bwd":
        ccr.ccr_rms_norm_bwd(ctx, st["dy"].unbind(), st["h"].unbind(), [st["w"]] * R, st["rstd"].unbind(),
                             st["dx"].unbind(), st["dw"].unbind(), st["work"],
                             dh=st["dh"].unbind() if case["add"] else None)
        return {"dx": st["dx"], "dw": st["dw"]}
    if op == "route":
        more, res = {}, {"topk": st["topk"], "weights": st["weights"]}
        if case["stats"]:
            more = dict(counts=st["counts"].unbind(), score_sums=st["sums"].unbind(), work=st["work"])
            res.update(counts=st["counts"], sums=st["sums"])
        ccr.ccr_moe_route(ctx, st["logits"].unbind(), st["topk"].unbind(), st["weights"].unbind(),
                          bias=[st["bias"]] * R if case["bias"] else None, score=case["score"],
                          groups=case["groups"], kept=case["kept"], group_top=case["group_top"],
                          renorm=case["renorm"], scale=case["scale"], **more)
        return res
    if op == "route_bwd":
        ccr.ccr_moe_route_bwd(ctx, st["logits"].unbind(), st["topk"].unbind(), st["dweights"].unbind(),
                              st["dlogits"].unbind(),
                              dscore_sums=st["dsums"].unbind() if case["stats"] else None,
                              score=case["score"], renorm=case["renorm"], scale=case["scale"])
        return st["dlogits"]
    if op == "quantize":
        ccr.ccr_quantize_rows(ctx, st["x"].unbind(), st["q"].unbind())
        ccr.ccr_dequantize_rows(ctx, st["q"].unbind(), st["values"].unbind())
        return st["values"]
    if op == "dequantize":
        ccr.ccr_dequantize_rows(ctx, st["q"].unbind(), st["values"].unbind())
        return st["values"]
    ccr.ccr_moe_experts_q8(ctx, _ranks(st["exp"], st["per_rank"]), st["w"].unflatten(0, (R, -1)).unbind(),
                           st["ecnt"], case["H"], _ranks(st["out"], st["per_rank"]))
    return st["out"]


# ----------------------------------------------------------- in 64 bits
def _grid8(y):
    """y [..., H] in 64 bits on the grid of rows of 8 bits, from the formula."""
    H = y.shape[-1]
    v = torch.zeros(*y.shape[:-1], -(-H // 32) * 32, dtype=torch.float64, device="cuda")
    v[..., :H] = y
    v = v.view(*y.shape[:-1], -1, 32)
    top = v.abs().amax(dim=-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448))
    e = torch.where(448 * torch.exp2(e - 1) >= top, e - 1, e)  # where the logarithm was rounded up
    e = torch.where(448 * torch.exp2(e) < top, e + 1, e).clamp(min=-127)
    q = v / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step * torch.exp2(e)).reshape(*y.shape[:-1], -1)[..., :H]


def exact(case, seed):
    """The operator's definition in 64 bits on the inputs of (case, seed)."""
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "norm":
        res = {}
        h = st["x"].to(f64)
        if case["add"]:  # h is held in the rows' type, and the norm is that of h
            h = h + st["res"].to(f64)
            res["h"] = h
            h = h.to(st["x"].dtype).to(f64)
        rstd = (torch.linalg.vector_norm(h, dim=-1) ** 2 / case["H"] + EPS) ** -0.5
        y = st["w"].to(f64) * h * rstd[:, :, None]
        if case["out"] != "q8":
            res["y"] = y
        if case["out"] != "y":
            res["values"] = _grid8(y)
        return {**res, "rstd": rstd}
    if op == "norm_bwd":
        h, r, w, dy = (st[k].to(f64) for k in ("h", "rstd", "w", "dy"))
        r = r[:, :, None]
        inner = torch.einsum("rth,rth,h->rt", dy, h, w)[:, :, None] / case["H"]
        dx = r * w * dy - r ** 3 * inner * h
        if case["add"]:
            dx = dx + st["dh"].to(f64)
        return {"dx": dx, "dw": torch.einsum("rth,rth->rh", dy, h * r)}
    if op in ("route", "route_bwd"):
        l = st["logits"].to(f64)
        sm = case["score"] == "softmax"
        s = torch.softmax(l, dim=-1) if sm else torch.sigmoid(l)
        if op == "route":
            chosen = _choose(case, st["logits"], st["bias"])[0]
        else:
            chosen = st["topk"].long()
        pick = torch.nn.functional.one_hot(chosen, case["E"]).to(f64)  # [R, T, K, E]
        c = (pick * s[:, :, None, :]).sum(dim=-1)
        if op == "route":
            w = case["scale"] * (c / c.sum(dim=-1, keepdim=True) if case["renorm"] else c)
            res = {"topk": None, "weights": w}
            if case["stats"]:
                res.update(counts=None, sums=s.sum(dim=1))
            return res
        # the Jacobian of the weights by the scores, then of the scores by the logits
        dw = st["dweights"].to(f64)
        if case["renorm"]:
            total = c.sum(dim=-1)
            back = dw / total[..., None] - ((dw * c).sum(dim=-1) / total ** 2)[..., None]
        else:
            back = dw
        ds = case["scale"] * (pick * back[..., None]).sum(dim=2)
        if case["stats"]:
            ds = ds + st["dsums"].to(f64)[:, None, :]
        return s * ds - s * (s * ds).sum(dim=-1, keepdim=True) if sm else ds * (s - s * s)
    if op == "quantize":
        return _grid8(st["x"].to(f64))
    H = case["H"]
    blocks = -(-H // 128)

    def values(rows):  # from the bytes: sign, 4 bits of exponent, 3 of mantissa
        b = rows[..., :blocks * 128].to(torch.int64)
        mant, ex = (b & 7).to(f64), (b >> 3) & 15
        mag = torch.where(ex == 0, mant * 2.0 ** -9, (8 + mant) * torch.exp2((ex - 10).to(f64)))
        v = torch.where(b >= 128, -mag, mag).unflatten(-1, (-1, 32))
        e = rows[..., blocks * 128:blocks * 132].to(f64) - 127
        return (v * torch.exp2(e)[..., None]).flatten(-2)[..., :H]

    if op == "dequantize":
        return values(st["q"])
    out = torch.zeros(sum(st["rows"]), case["F"], dtype=f64, device="cuda")
    at = 0
    for e, n in enumerate(st["rows"]):  # out[i, f] = sum_h exp[i, h] w[f, h]
        if n:
            out[at:at + n] = torch.mm(values(st["w"][e]), values(st["exp"][at:at + n]).T).T
        at += n
    return out
