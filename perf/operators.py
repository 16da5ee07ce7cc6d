"""Cases for the training- and serving-step operators around the MoE exchange
and the gradient buckets:

  experts, dgrad, wgrad   the experts' matrix products on dispatched rows,
                          ragged by expert, and their two gradients
  gate, gate_bwd          the softmax of the router's chosen logits applied to
                          the K returned rows of each token, and its gradients
  norm, clip              the global 2-norm over many gradient tensors, and
                          clipping to a maximum norm

With ``own`` false, ``run`` computes an operator in elementary torch
operations; with ``own`` true it calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # One training layer at the expert-parallel dispatch workload's size: 8
        # ranks x 4096 tokens x top 6 of 64 experts, hidden 2048, popular and
        # unpopular experts; the product that follows the dispatch.
        dict(name="experts_train_bf16", op="experts", dtype="bf16", R=8, T=4096, E=64, K=6,
             H=2048, F=1024, skew=0.5, route=11),
        # The same layer on two ranks with an expert width that is no multiple
        # of a tile: the gradient of the dispatched rows ...
        dict(name="dgrad_train_bf16", op="dgrad", dtype="bf16", R=2, T=4096, E=16, K=6,
             H=2048, F=1408, skew=0.5, route=12),
        # ... and of the experts' weights, in fp32 as an optimizer keeps them.
        dict(name="wgrad_train_bf16_f32", op="wgrad", dtype="bf16", out="f32", R=2, T=4096, E=16,
             K=6, H=2048, F=1408, skew=0.5, route=13),
        # A small fp32 layer with odd sizes, some experts without a row.
        dict(name="experts_odd_f32", op="experts", dtype="f32", R=2, T=700, E=24, K=2,
             H=1036, F=500, skew=1.5, route=14),
        # Serving: one token through its six experts; the weights are the work.
        dict(name="experts_token_bf16", op="experts", dtype="bf16", R=1, T=1, E=64, K=6,
             H=2048, F=1024, skew=0.0, route=15),
        # Serving: a decode batch of 48 tokens over all 64 experts, few rows each.
        dict(name="experts_batch_bf16", op="experts", dtype="bf16", R=1, T=48, E=64, K=6,
             H=2048, F=1024, skew=0.5, route=16),
        # The weighted sum that ends the layer, at the dispatch workload's size.
        dict(name="gate_train_bf16", op="gate", dtype="bf16", R=8, T=4096, E=64, K=6,
             H=2048, norm="chosen", drop=0),
        # Its gradients on one rank, softmax over all experts, some choices dropped
        # by a capacity limit.
        dict(name="gate_bwd_train_bf16", op="gate_bwd", dtype="bf16", R=2, T=4096, E=64, K=6,
             H=2048, norm="all", drop=6),
        # Serving: the weighted sum of one token.
        dict(name="gate_token_bf16", op="gate", dtype="bf16", R=1, T=1, E=64, K=6,
             H=2048, norm="chosen", drop=0),
        # The global norm over one data-parallel bucket's worth of bf16 gradients
        # (25 Mi values) in 150 tensors, packed back to back at element offsets.
        dict(name="norm_bucket_bf16", op="norm", types="bf16", n=150, total=25 << 20,
             scale=1e-3, packed=True, route=21),
        # Clipping a shard's gradients, 200 Mi values in 300 tensors of both types.
        dict(name="clip_shard_mixed", op="clip", types="mixed", n=300, total=200 << 20,
             scale=1e-3, packed=False, max_norm=1.0, route=22),
        # Clipping the few small tensors of norms and biases: latency.
        dict(name="clip_small_f32", op="clip", types="f32", n=24, total=40000,
             scale=0.1, packed=True, max_norm=1.0, route=23),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["experts", "experts", "dgrad", "wgrad", "gate", "gate_bwd", "norm", "clip"])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    route = rng.randrange(1 << 30)
    if op in ("experts", "dgrad", "wgrad"):
        R = rng.choice([1, 1, 2, 4, 8])
        E = R * rng.choice([1, 2, 3, 4, 8])
        K = rng.randint(1, min(E, 8))
        H = 8 * _log(rng, 8, 512)
        F = 8 * _log(rng, 8, 512)
        T = _log(rng, 1, 8192)
        # at most a third of the largest listed case's flops (fp32: a thirtieth)
        top = 0.27e12 if dt == "bf16" else 0.027e12
        T = max(1, min(T, int(top / (2.0 * R * K * H * F))))
        case = dict(op=op, dtype=dt, R=R, T=T, E=E, K=K, H=H, F=F,
                    skew=rng.choice([0.0, 0.5, 1.5]), route=route)
        if op == "wgrad":
            case["out"] = rng.choice(["f32", dt])
        return case
    if op in ("gate", "gate_bwd"):
        R = rng.choice([1, 2, 4, 8])
        E = rng.choice([4, 8, 16, 60, 64, 128, 256])
        K = rng.randint(1, min(E, 8))
        H = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, 8192)
        T = max(1, min(T, int(0.4e9 / (R * K * H * SIZE[dt]))))
        return dict(op=op, dtype=dt, R=R, T=T, E=E, K=K, H=H, norm=rng.choice(["chosen", "all"]),
                    drop=rng.choice([0, 0, 6, 40]))
    n = _log(rng, 1, 600)
    case = dict(op=op, types=rng.choice(["bf16", "f32", "mixed"]), n=n,
                total=max(n, _log(rng, 1000, 100 << 20)), scale=rng.choice([1e-3, 0.1]),
                packed=rng.random() < 0.5, route=route)
    if op == "clip":
        case["max_norm"] = rng.choice([0.5, 1.0, 1e9])
    return case


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


def tensor_sizes(case):
    """(elements, type name) of each gradient tensor: lengths spread over two
    orders of magnitude around total / n, most of them odd."""
    rng = random.Random(case["route"])
    w = [math.exp(rng.uniform(-2.5, 2.5)) for _ in range(case["n"])]
    s = sum(w)
    out = []
    for x in w:
        dt = rng.choice(["bf16", "f32"]) if case["types"] == "mixed" else case["types"]
        out.append((max(1, int(case["total"] * x / s)), dt))
    return out


def absent_choices(case):
    """bool [T, K]: choices that a capacity limit dropped (their topk entry is -1)."""
    i = np.arange(case["T"] * case["K"], dtype=np.int64)
    return ((i * 7919 % 100) < case["drop"]).reshape(case["T"], case["K"])


def work(case):
    op = case["op"]
    if op in ("experts", "dgrad", "wgrad"):
        rows = expert_rows(case)
        n, used = int(rows.sum()), int((rows > 0).sum())
        H, F, s = case["H"], case["F"], SIZE[case["dtype"]]
        wbytes = case["E"] * H * F * SIZE[case["out"]] if op == "wgrad" else used * H * F * s
        return {"bytes": n * (H + F) * s + wbytes, "flops": 2 * n * H * F}
    if op in ("gate", "gate_bwd"):
        R, T, E, K, H, s = (case["R"], case["T"], case["E"], case["K"], case["H"], SIZE[case["dtype"]])
        kept = T * K - int(absent_choices(case).sum())
        small = T * K * 4 + (T * E * 4 if case["norm"] == "all" else kept * 4)
        if op == "gate":
            return {"bytes": R * (kept * H * s + T * H * s + small), "flops": R * 2 * kept * H}
        return {"bytes": R * (kept * H * s + T * H * s + small + T * K * H * s + T * E * 4),
                "flops": R * 3 * kept * H}
    sizes = tensor_sizes(case)
    nbytes, n = sum(c * SIZE[t] for c, t in sizes), sum(c for c, _ in sizes)
    if op == "norm":
        return {"bytes": nbytes + 4, "flops": 2 * n}
    return {"bytes": 2 * nbytes + 4, "flops": 3 * n}


# ------------------------------------------------------------------ inputs
def _normal(g, shape, scale, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _carve(case, make):
    """(flat, views): one flat buffer per type, make(type, elements), and each
    tensor's view of it: packed back to back at element offsets, or each at a
    multiple of 8 elements."""
    sizes = tensor_sizes(case)
    step = 1 if case["packed"] else 8
    room = {}
    for c, t in sizes:
        room[t] = room.get(t, 0) + -(-c // step) * step
    flat = {t: make(t, room[t]) for t in sorted(room)}
    at, views = dict.fromkeys(flat, 0), []
    for c, t in sizes:
        views.append(flat[t][at[t]:at[t] + c])
        at[t] += -(-c // step) * step
    return flat, views


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("experts", "dgrad", "wgrad"):
        dt = DT[case["dtype"]]
        R, E, H, F = case["R"], case["E"], case["H"], case["F"]
        rows = expert_rows(case)
        st["ecnt"], st["rows"] = expert_counts(case), rows.tolist()
        tot = [int(rows[d].sum()) for d in range(R)]
        if op != "dgrad":
            st["exp"] = [_normal(g, (t, H), 1.0, dt) for t in tot]
        if op != "experts":
            st["dout"] = [_normal(g, (t, F), 0.02, dt) for t in tot]
        if op != "wgrad":
            st["w"] = [_normal(g, (E // R, F, H), 1.0 / math.sqrt(H), dt) for _ in range(R)]
        shape = {"experts": lambda t: (t, F), "dgrad": lambda t: (t, H),
                 "wgrad": lambda t: (E // R, F, H)}[op]
        odt = DT[case["out"]] if op == "wgrad" else dt
        st["out"] = [torch.empty(shape(t), dtype=odt, device="cuda") for t in tot]
    elif op in ("gate", "gate_bwd"):
        dt = DT[case["dtype"]]
        R, T, E, K, H = case["R"], case["T"], case["E"], case["K"], case["H"]
        gone = torch.from_numpy(absent_choices(case)).cuda()
        st["rows"] = [_normal(g, (T, K, H), 1.0, dt) for _ in range(R)]
        st["logits"] = [_normal(g, (T, E), 1.5, torch.float32) for _ in range(R)]
        st["topk"] = [torch.where(gone, -1, torch.topk(l, K, dim=1).indices).to(torch.int32)
                      for l in st["logits"]]
        if op == "gate":
            st["y"] = [torch.empty(T, H, dtype=dt, device="cuda") for _ in range(R)]
        else:
            st["dy"] = [_normal(g, (T, H), 0.02, dt) for _ in range(R)]
            st["drows"] = [torch.empty(T, K, H, dtype=dt, device="cuda") for _ in range(R)]
            st["dlogits"] = [torch.empty(T, E, dtype=torch.float32, device="cuda") for _ in range(R)]
    else:
        def values(t, count):
            return _normal(g, (count,), case["scale"], DT[t])

        st["grads"] = _carve(case, values)[1]
        if op == "clip":  # the clipped gradients go to buffers of their own
            st["flat"], st["out"] = _carve(case, lambda t, count: torch.zeros(count, dtype=DT[t], device="cuda"))
        st["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
    if own:
        import collective_communication_reduce_amd as ccr
        st["ctx"] = ccr.Context(torch.cuda.current_device())
        if op in ("norm", "clip"):
            st["work"] = torch.empty(ccr.CCR_GRAD_WORK, dtype=torch.float64, device="cuda")
    return st


# ------------------------------------------------------------- plain forms
def _gate_weights(case, logits, topk):
    """(w [T, K], p [T, E]): the weights of the chosen experts, 0 where the choice
    is absent, and the softmax over the experts it is taken over."""
    have = topk >= 0
    at = topk.clamp(min=0).long()
    ninf = float("-inf")
    if case["norm"] == "chosen":
        l = torch.where(have, logits.gather(1, at), torch.full((), ninf, device=logits.device))
        top = l.max(dim=1, keepdim=True).values
        e = torch.where(l == ninf, torch.zeros_like(l), torch.exp(l - top))
        s = e.sum(dim=1, keepdim=True)
        return torch.where(s == 0, s, e / s), None
    top = logits.max(dim=1, keepdim=True).values
    e = torch.where(logits == ninf, torch.zeros_like(logits), torch.exp(logits - top))
    s = e.sum(dim=1, keepdim=True)
    p = torch.where(s == 0, s, e / s)
    return torch.where(have, p.gather(1, at), torch.zeros((), device=p.device)), p


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op in ("experts", "dgrad", "wgrad"):
        outs = []
        for d in range(case["R"]):
            at, parts = 0, []
            for l, n in enumerate(st["rows"][d]):
                sl = slice(at, at + n)
                at += n
                if op == "experts":
                    parts.append(st["exp"][d][sl].float() @ st["w"][d][l].float().t())
                elif op == "dgrad":
                    parts.append(st["dout"][d][sl].float() @ st["w"][d][l].float())
                else:
                    parts.append((st["dout"][d][sl].float().t() @ st["exp"][d][sl].float()).to(DT[case["out"]]))
            if op == "wgrad":
                outs.append(torch.stack(parts))
            else:
                outs.append(torch.cat(parts).to(DT[case["dtype"]]))
        return outs
    if op == "gate":
        outs = []
        for rows, logits, topk in zip(st["rows"], st["logits"], st["topk"]):
            w, _ = _gate_weights(case, logits, topk)
            kept = torch.where((topk >= 0)[:, :, None], rows.float(), torch.zeros((), device=rows.device))
            outs.append((w[:, :, None] * kept).sum(dim=1).to(rows.dtype))
        return outs
    if op == "gate_bwd":
        drows, dlogits = [], []
        for dy, rows, logits, topk in zip(st["dy"], st["rows"], st["logits"], st["topk"]):
            w, p = _gate_weights(case, logits, topk)
            have = topk >= 0
            dyf = dy.float()
            drows.append((w[:, :, None] * dyf[:, None, :]).to(rows.dtype))
            dw = (rows.float() * dyf[:, None, :]).sum(dim=2)
            dw = torch.where(have, dw, torch.zeros_like(dw))
            s = (w * dw).sum(dim=1, keepdim=True)
            own_part = torch.where(have, w * (dw - s) if p is None else w * dw, torch.zeros_like(dw))
            dl = torch.zeros_like(logits) if p is None else -p * s
            dlogits.append(dl.scatter_add(1, topk.clamp(min=0).long(), own_part))
        return {"drows": drows, "dlogits": dlogits}
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for x in st["grads"]:
        total = total + x.float().double().square().sum()
    norm = total.sqrt().float().reshape(1)
    if op == "norm":
        return norm
    scale = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)
    for x, o in zip(st["grads"], st["out"]):
        torch.mul(x.float(), scale, out=o)
    return {"norm": norm, "out": st["flat"]}


def run(state):
    if not own:
        return _plain(state)
    import collective_communication_reduce_amd as ccr
    st, case, op, ctx = state, state["case"], state["case"]["op"], state["ctx"]
    if op == "experts":
        ccr.ccr_moe_experts(ctx, st["exp"], st["w"], st["ecnt"], st["out"])
        return st["out"]
    if op == "dgrad":
        ccr.ccr_moe_experts_dgrad(ctx, st["dout"], st["w"], st["ecnt"], st["out"])
        return st["out"]
    if op == "wgrad":
        ccr.ccr_moe_experts_wgrad(ctx, st["exp"], st["dout"], st["ecnt"], st["out"])
        return st["out"]
    if op == "gate":
        ccr.ccr_moe_gate_sum(ctx, st["rows"], st["logits"], st["topk"], st["y"], norm=case["norm"])
        return st["y"]
    if op == "gate_bwd":
        ccr.ccr_moe_gate_sum_bwd(ctx, st["dy"], st["rows"], st["logits"], st["topk"], st["drows"],
                                 st["dlogits"], norm=case["norm"])
        return {"drows": st["drows"], "dlogits": st["dlogits"]}
    if op == "norm":
        ccr.ccr_grad_norm(ctx, st["grads"], st["work"], st["norm"])
        return st["norm"]
    ccr.ccr_grad_clip(ctx, st["grads"], case["max_norm"], st["work"], st["norm"], out=st["out"])
    return {"norm": st["norm"], "out": st["flat"]}


# ----------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The operator's definition in 64 bits on the inputs of (case, seed)."""
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op in ("experts", "dgrad", "wgrad"):
        res = []
        for d, rows in enumerate(st["rows"]):
            first = np.concatenate([[0], np.cumsum(rows)])
            n = int(first[-1])
            if op == "wgrad":
                out = torch.zeros(len(rows), case["F"], case["H"], dtype=f64, device="cuda")
            else:
                out = torch.zeros(n, case["F"] if op == "experts" else case["H"], dtype=f64, device="cuda")
            for e in range(len(rows)):
                lo, hi = int(first[e]), int(first[e + 1])
                if lo == hi:
                    continue
                if op == "experts":  # out[i, f] = sum_h exp[i, h] w[f, h]
                    out[lo:hi] = torch.mm(st["w"][d][e].to(f64), st["exp"][d][lo:hi].to(f64).T).T
                elif op == "dgrad":  # dexp[i, h] = sum_f dout[i, f] w[f, h]
                    out[lo:hi] = torch.mm(st["w"][d][e].to(f64).T, st["dout"][d][lo:hi].to(f64).T).T
                else:  # dw[f, h] = sum_i dout[i, f] exp[i, h]
                    out[e] = torch.mm(st["exp"][d][lo:hi].to(f64).T, st["dout"][d][lo:hi].to(f64)).T
            res.append(out)
        return res
    if op in ("gate", "gate_bwd"):
        ys, drs, dls = [], [], []
        for r in range(case["R"]):
            l, top = st["logits"][r].to(f64), st["topk"][r]
            T, E = l.shape
            K = top.shape[1]
            pick = torch.zeros(T, K, E, dtype=f64, device="cuda")  # one-hot of each kept choice
            t, k = torch.nonzero(top >= 0, as_tuple=True)
            pick[t, k, top[t, k].long()] = 1.0
            z = torch.exp(l - l.amax(dim=1, keepdim=True))
            if case["norm"] == "chosen":
                z = z * pick.sum(dim=1)
            zs = z.sum(dim=1, keepdim=True)
            p = z / torch.where(zs > 0, zs, torch.ones_like(zs))
            w = (pick * p[:, None, :]).sum(dim=2)
            x = st["rows"][r].to(f64) * (top >= 0).to(f64)[:, :, None]
            if op == "gate":
                y = torch.zeros(T, case["H"], dtype=f64, device="cuda")
                for k in range(K):
                    y += w[:, k, None] * x[:, k]
                ys.append(y)
                continue
            dy = st["dy"][r].to(f64)
            drs.append(torch.stack([w[:, k, None] * dy for k in range(K)], dim=1))
            dp = torch.zeros(T, E, dtype=f64, device="cuda")
            for k in range(K):
                dp += pick[:, k] * (x[:, k] * dy).sum(dim=1, keepdim=True)
            dls.append(p * (dp - (p * dp).sum(dim=1, keepdim=True)))
        return ys if op == "gate" else {"drows": drs, "dlogits": dls}
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(x.to(f64))) ** 2 for x in st["grads"]))
    as_tensor = torch.tensor([norm], dtype=f64, device="cuda")
    if op == "norm":
        return as_tensor
    c = min(1.0, case["max_norm"] / (norm + 1e-6))
    flat, out = _carve(case, lambda t, count: torch.zeros(count, dtype=f64, device="cuda"))
    for x, o in zip(st["grads"], out):
        o.copy_(x.to(f64) * c)
    return {"norm": as_tensor, "out": flat}
