"""The front of an expert-parallel layer as a training program runs it: residual
and norm, the router, 8-bit rows through the exchange, the products on them, the
sum by the router's weights, and the way back, against autograd in 64 bits."""
import numpy as np
import pytest

import rows8_helpers as r8
from gpu_helpers import say, torch_cuda
from operator_helpers import HALF

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


@pytest.mark.parametrize("R,T,E,K,H,F", [(2, 40, 8, 3, 64, 136), (4, 130, 16, 4, 264, 72), (1, 1, 4, 2, 32, 48)])
@pytest.mark.parametrize("score,groups,kept", [("softmax", 1, 1), ("sigmoid", 4, 2)])
def test_training_step(ccr_mod, R, T, E, K, H, F, score, groups, kept):
    import torch
    ccr = ccr_mod
    say(f"moe front R={R} T={T} E={E} K={K} H={H} F={F} {score}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, res = [rnd(T, H) for _ in range(R)], [rnd(T, H) for _ in range(R)]
    gain, wr = 1 + 0.1 * rnd(H), rnd(E, H) / H ** 0.5
    w = [rnd(E // R, F, H) / H ** 0.5 for _ in range(R)]
    bias, dy, dh = 0.05 * rnd(E), [rnd(T, F) for _ in range(R)], [rnd(T, H) for _ in range(R)]
    dsum = 0.1 * rnd(E)
    how = dict(score=score, renorm=True, scale=1.5)
    B = ccr.ccr_q8_row_bytes(H)
    with ccr.Context(0) as c:
        h, y = ([torch.zeros(T, H, **f32) for _ in range(R)] for _ in range(2))
        q, rstd = [torch.zeros(T, B, **u8) for _ in range(R)], [torch.zeros(T, **f32) for _ in range(R)]
        ccr.ccr_rms_norm(c, x, [gain] * R, y=y, q=q, residual=res, h=h, rstd=rstd)
        logits = [a @ wr.t() for a in y]
        topk, gate = [torch.zeros(T, K, **i32) for _ in range(R)], [torch.zeros(T, K, **f32) for _ in range(R)]
        counts = [torch.zeros(E, dtype=torch.int64, device="cuda") for _ in range(R)]
        sums = [torch.zeros(E, **f32) for _ in range(R)]
        rwork = torch.empty(ccr.ccr_moe_route_work(R, T, E), **f32)
        ccr.ccr_moe_route(c, logits, topk, gate, bias=[bias] * R, groups=groups, kept=kept, group_top=2, counts=counts,
                          score_sums=sums, work=rwork, **how)
        src_tok, slot = ([torch.zeros(T * K, **i32) for _ in range(R)] for _ in range(2))
        ecnt = np.stack([ccr.ccr_moe_plan(c, topk[r], E, R, src_tok[r], slot[r]) for r in range(R)])
        assert np.array_equal(ecnt, torch.stack(counts).cpu().numpy())
        rows = [int(n) for n in ecnt.sum(axis=0).reshape(R, -1).sum(axis=1)]
        # 8-bit rows through the exchange (staged and fused give the same), products
        exp8 = [torch.zeros(n, B, **u8) for n in rows]
        ccr.ccr_moe_dispatch_fused(c, q, src_tok, ecnt, K, exp8)
        send, recv, again = ([torch.zeros(m, B, **u8) for m in n] for n in ([T * K] * R, rows, rows))
        ccr.ccr_moe_dispatch(c, q, src_tok, ecnt, K, send, recv, again)
        w8 = [torch.zeros(E // R, F, B, **u8) for _ in range(R)]
        ccr.ccr_quantize_rows(c, w, w8)
        mid16 = [torch.zeros(n, F, dtype=torch.bfloat16, device="cuda") for n in rows]
        ccr.ccr_moe_experts_q8(c, exp8, w8, ecnt, H, mid16)
        # the same rows and weights in fp32, for the rest of the step
        exp, wq = [torch.zeros(n, H, **f32) for n in rows], [torch.zeros_like(v) for v in w]
        ccr.ccr_dequantize_rows(c, exp8, exp)
        ccr.ccr_dequantize_rows(c, w8, wq)
        mid, back = [torch.zeros(n, F, **f32) for n in rows], [torch.zeros(T, K, F, **f32) for _ in range(R)]
        ccr.ccr_moe_experts(c, exp, wq, ecnt, mid)
        ccr.ccr_moe_combine_fused(c, mid, slot, ecnt, T, K, back)
        out = [torch.zeros(T, F, **f32) for _ in range(R)]
        ccr.ccr_moe_gate_sum(c, back, gate, topk, out, norm="given")
        # backward
        dback, dgate = [torch.zeros(T, K, F, **f32) for _ in range(R)], [torch.zeros(T, K, **f32) for _ in range(R)]
        ccr.ccr_moe_gate_sum_bwd(c, dy, back, gate, topk, dback, dgate, norm="given")
        dl = [torch.zeros(T, E, **f32) for _ in range(R)]
        ccr.ccr_moe_route_bwd(c, logits, topk, dgate, dl, dscore_sums=[dsum] * R, **how)
        choice = [torch.argsort(s.long()).to(torch.int32) for s in slot]
        dmid, dexp = [torch.zeros(n, F, **f32) for n in rows], [torch.zeros(n, H, **f32) for n in rows]
        ccr.ccr_moe_dispatch_fused(c, [d.view(T * K, F) for d in dback], choice, ecnt, 1, dmid)
        ccr.ccr_moe_experts_dgrad(c, dmid, wq, ecnt, dexp)
        dw = [torch.zeros(E // R, F, H, **f32) for _ in range(R)]
        ccr.ccr_moe_experts_wgrad(c, exp, dmid, ecnt, dw)
        dyk = [torch.zeros(T, K, H, **f32) for _ in range(R)]
        ccr.ccr_moe_combine_fused(c, dexp, slot, ecnt, T, K, dyk)
        dnorm = [dyk[r].sum(1) + dl[r] @ wr for r in range(R)]
        dx, dgain = [torch.zeros(T, H, **f32) for _ in range(R)], [torch.zeros(H, **f32) for _ in range(R)]
        nwork = torch.empty(ccr.ccr_rms_norm_work(R, T, H), **f32)
        ccr.ccr_rms_norm_bwd(c, dnorm, h, [gain] * R, rstd, dx, dgain, nwork, dh=dh)
        shared = [d.clone() for d in dgain]
        if R > 1:
            ccr.ccr_allreduce(c, shared)  # the ranks' parts of the shared weight's gradient
        torch.cuda.synchronize()
    for a, b in zip(exp8, again):
        assert torch.equal(a, b)
    # products on 8-bit rows: the fp32 products of what they stand for, within the
    # instruction's alignment (16 products to 2^-13 of the largest) and a bf16 rounding
    for a, b, e in zip(mid16, mid, exp):
        bound = 16 * 2.0 ** -13 * (H / 16) * float(e.abs().max()) * float(max(v.abs().max() for v in wq)) if len(e) else 0
        assert bool(((a.double() - b.double()).abs() <= HALF["bf16"] * b.double().abs() + bound).all())
    # the same layer in float64 through autograd, with the choices held and rounding
    # to 8 bits passed through as it is
    D = lambda ts: torch.cat([t.double().cpu() for t in ts])
    X = (D(x) + D(res)).requires_grad_()
    G, W = gain.double().cpu().requires_grad_(), D(w).requires_grad_()
    Wq = W + (D(wq) - D(w))
    N = X * (X.square().mean(1, keepdim=True) + 1e-6).rsqrt() * G
    values = torch.from_numpy(np.concatenate([r8.unpack(t.cpu().numpy(), H)[0] for t in q]))
    Nq = N + (values - N).detach()
    L = N @ wr.double().cpu().t()
    S = L.softmax(1) if score == "softmax" else L.sigmoid()
    pick = torch.cat(topk).long().cpu()
    P = S.gather(1, pick)
    P = 1.5 * P / P.sum(1, keepdim=True)
    Y = sum(P[:, k:k + 1] * (Wq[pick[:, k]] * Nq[:, None, :]).sum(-1) for k in range(K))
    ((Y * D(dy)).sum() + (X * D(dh)).sum() + (S * dsum.double().cpu()).sum()).backward()

    def near(got, want, terms):
        # every value is a sum of at most `terms` products of fp32 values, each
        # product carrying the roundings of at most 400 operations
        scale = float(want.abs().max()) or 1.0
        err = float((got.double().cpu() - want).abs().max())
        assert err <= (terms + 400) * U * scale * 8, (err, scale)

    assert bool((torch.cat(sums).view(R, E).sum(0).double().cpu() - S.sum(0).detach()).abs().max() <= (T + 400) * U * T * R)
    near(torch.cat(out), Y.detach(), H + K)
    near(torch.cat(dx), X.grad, H + F + E + K)
    near(torch.cat(dw), W.grad, R * T + K)
    near(sum(dgain), G.grad, R * T + H + F + E)
    if R > 1:
        assert all(torch.equal(s, shared[0]) for s in shared)
        near(shared[0], G.grad, R * T + H + F + E)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,H", [(1, 6, 2048), (33, 3, 24), (7, 16, 520), (130, 1, 4096), (9, 8, 136)])
def test_gate_sum_with_given_weights(ccr_mod, T, K, H, dt):
    """y, drows and the weights' gradients against 64 bits; absent choices (ids
    outside the range) are not read, weighted or given a gradient."""
    import torch
    from operator_helpers import Guarded, inside_nan, tdtype
    say(f"gate given T={T} K={K} H={H} {dt}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T * K)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    rows = rnd(T, K, H).to(tdtype(dt))
    w = rnd(T, K)
    topk = torch.randint(0, 1024, (T, K), generator=g, device="cuda", dtype=torch.int32)
    gone = torch.rand(T, K, generator=g, device="cuda") < 0.3
    topk[gone] = -1
    topk[T - 1, K - 1] = 1024
    gone[T - 1, K - 1] = True
    rows[gone] = float("nan")
    w[gone] = float("nan")
    dy = inside_nan(rnd(T, H).to(tdtype(dt)))
    rows, w = inside_nan(rows), inside_nan(w)
    y, dr, dw = Guarded((T, H), tdtype(dt)), Guarded((T, K, H), tdtype(dt)), Guarded((T, K), torch.float32)
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_gate_sum(c, [rows], [w], [topk], [y.t], norm="given")
        ccr_mod.ccr_moe_gate_sum_bwd(c, [dy], [rows], [w], [topk], [dr.t], [dw.t], norm="given")
        torch.cuda.synchronize()
    assert y.intact() and dr.intact() and dw.intact()
    have = ~gone[:, :, None]
    ww, x = torch.where(have[:, :, 0], w.double(), 0.0)[:, :, None], torch.where(have, rows.double(), 0.0)
    want, mag = (ww * x).sum(1), (ww * x).abs().sum(1)
    assert bool(((y.t.double() - want).abs() <= HALF[dt] * want.abs() + (K + 1) * U * mag).all())
    want = ww * dy.double()[:, None]
    assert bool(((dr.t.double() - want).abs() <= (HALF[dt] + 1.01 * U) * want.abs()).all())
    p = x * dy.double()[:, None]
    # a thread adds at most H / 64 + 8 products, then waves and the workgroup
    assert bool(((dw.t.double() - p.sum(2)).abs() <= (H // 64 + 8 + 12) * U * p.abs().sum(2)).all())
    assert not bool(dw.t[gone].any()) and not bool(dr.t[gone].any())
