"""One expert-parallel layer forward and backward, its weight gradients summed
over data-parallel replicas, measured and clipped: every call of the step in
the order a training program makes them, against the formulas in 64 bits."""
import numpy as np
import pytest

from gpu_helpers import say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


@pytest.mark.parametrize("R,T,E,K,H,F", [(2, 40, 8, 3, 64, 136), (4, 130, 16, 4, 264, 72), (1, 1, 4, 2, 32, 48)])
@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_training_step(ccr_mod, R, T, E, K, H, F, norm):
    import torch
    ccr = ccr_mod
    say(f"moe layer R={R} T={T} E={E} K={K} H={H} F={F} {norm}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    f32 = dict(dtype=torch.float32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = [rnd(T, H) for _ in range(R)]
    logits = [rnd(T, E) for _ in range(R)]
    dy = [rnd(T, F) for _ in range(R)]
    w = [rnd(E // R, F, H) / H ** 0.5 for _ in range(R)]
    with ccr.Context(0) as c:
        topk = [torch.zeros(T, K, **i32) for _ in range(R)]
        src_tok = [torch.zeros(T * K, **i32) for _ in range(R)]
        slot = [torch.zeros(T * K, **i32) for _ in range(R)]
        ecnt = []
        for r in range(R):
            ccr.ccr_moe_topk(c, logits[r], topk[r])
            ecnt.append(ccr.ccr_moe_plan(c, topk[r], E, R, src_tok[r], slot[r]))
        ecnt = np.stack(ecnt)
        rows = [int(n) for n in ecnt.sum(axis=0).reshape(R, -1).sum(axis=1)]
        # forward: dispatch, products, combine, gated sum
        exp = [torch.zeros(n, H, **f32) for n in rows]
        mid = [torch.zeros(n, F, **f32) for n in rows]
        back = [torch.zeros(T, K, F, **f32) for _ in range(R)]
        y = [torch.zeros(T, F, **f32) for _ in range(R)]
        ccr.ccr_moe_dispatch_fused(c, x, src_tok, ecnt, K, exp)
        ccr.ccr_moe_experts(c, exp, w, ecnt, mid)
        ccr.ccr_moe_combine_fused(c, mid, slot, ecnt, T, K, back)
        ccr.ccr_moe_gate_sum(c, back, logits, topk, y, norm=norm)
        # backward: the rows' gradients go to their experts as T*K tokens of one choice each
        dback = [torch.zeros(T, K, F, **f32) for _ in range(R)]
        dlogits = [torch.zeros(T, E, **f32) for _ in range(R)]
        ccr.ccr_moe_gate_sum_bwd(c, dy, back, logits, topk, dback, dlogits, norm=norm)
        choice = [torch.argsort(s.long()).to(torch.int32) for s in slot]
        dmid = [torch.zeros(n, F, **f32) for n in rows]
        ccr.ccr_moe_dispatch_fused(c, [d.view(T * K, F) for d in dback], choice, ecnt, 1, dmid)
        dexp = [torch.zeros(n, H, **f32) for n in rows]
        dw = [torch.zeros(E // R, F, H, **f32) for _ in range(R)]
        ccr.ccr_moe_experts_dgrad(c, dmid, w, ecnt, dexp)
        ccr.ccr_moe_experts_wgrad(c, exp, dmid, ecnt, dw)
        dback_x = [torch.zeros(T, K, H, **f32) for _ in range(R)]
        ccr.ccr_moe_combine_fused(c, dexp, slot, ecnt, T, K, dback_x)
        # two data-parallel replicas of rank 0's weights with the same gradient
        pair = [dw[0].clone(), dw[0].clone()]
        ccr.ccr_allreduce(c, pair)
        work = torch.empty(ccr.CCR_GRAD_WORK, dtype=torch.float64, device="cuda")
        total = torch.empty(1, **f32)
        clipped = [torch.empty_like(pair[0])] + [torch.empty_like(d) for d in dlogits]
        ccr.ccr_grad_clip(c, [pair[0]] + dlogits, 0.5, work, total, out=clipped)
        torch.cuda.synchronize()
    # the same layer in float64 through autograd, on the CPU
    W = torch.cat(w).double().cpu().requires_grad_()
    L = torch.cat(logits).double().cpu().requires_grad_()
    X = torch.cat(x).double().cpu().requires_grad_()
    pick = torch.cat(topk).long().cpu()
    l = L.gather(1, pick)
    p = l.softmax(1) if norm == "chosen" else L.softmax(1).gather(1, pick)
    Y = sum(p[:, k:k + 1] * (W[pick[:, k]] * X[:, None, :]).sum(-1) for k in range(K))
    (Y * torch.cat(dy).double().cpu()).sum().backward()

    def near(got, want, terms):
        # every value is a sum of at most `terms` products of fp32 values, each
        # product carrying the roundings of at most 200 operations
        scale = float(want.abs().max()) or 1.0
        err = float((got.double().cpu() - want).abs().max())
        assert err <= (terms + 200) * 2.0 ** -24 * scale * 8, (err, scale)

    near(torch.cat(y), Y.detach(), H + K)
    near(torch.cat(dback_x).sum(1), X.grad, F + K)
    near(torch.cat(dlogits), L.grad, H + F + K)
    near(torch.cat(dw), W.grad, R * T + K)
    near(pair[0], 2 * W.grad[:E // R], R * T + K)
    gsum = torch.sqrt((4 * W.grad[:E // R] ** 2).sum() + (L.grad ** 2).sum())
    near(total, gsum.reshape(1), R * T + K + H + F)
    near(clipped[0], 2 * W.grad[:E // R] * min(1.0, 0.5 / (float(gsum) + 1e-6)), R * T + K + H + F)


def test_tokens_and_experts_that_a_call_would_not_compute_are_refused(ccr_mod):
    """A rank with more (or fewer) tokens than the first, in any buffer, and more
    weights than the ranks' experts: refused, and nothing written."""
    import torch
    dev = dict(device="cuda")
    T, K, H, E = 3, 2, 8, 4

    def gate(n):
        return [torch.ones(n, K, H, **dev), torch.ones(n, E, **dev), torch.zeros(n, K, dtype=torch.int32, **dev),
                torch.ones(n, H, **dev), torch.full((n, K, H), 7.0, **dev), torch.full((n, E), 7.0, **dev),
                torch.full((n, H), 7.0, **dev)]

    first = gate(T)
    with ccr_mod.Context(0) as c:
        for n in (T - 1, T + 1):
            for i in range(7):  # the second rank's i-th buffer, or all of them
                second = gate(T)
                second[i] = gate(n)[i]
                for other in (second, gate(n)):
                    rows, logits, topk, dy, dr, dl, y = ([a, b] for a, b in zip(first, other))
                    if i in (0, 1, 2, 6) or other is not second:
                        with pytest.raises(ValueError, match="shape"):
                            ccr_mod.ccr_moe_gate_sum(c, rows, logits, topk, y)
                    if i != 6 or other is not second:
                        with pytest.raises(ValueError, match="shape"):
                            ccr_mod.ccr_moe_gate_sum_bwd(c, dy, rows, logits, topk, dr, dl)
                    torch.cuda.synchronize()
                    assert all(bool((t == 7.0).all()) for t in (*dr, *dl, *y))
        x, y = torch.ones(5, H, **dev), torch.full((5, 16), 7.0, **dev)
        ecnt = [[1, 2, 0, 0]]
        for experts in (3, 5):
            w = torch.full((experts, 16, H), 7.0, **dev)
            with pytest.raises(ValueError, match="shape"):
                ccr_mod.ccr_moe_experts(c, [x], [w], ecnt, [y])
            with pytest.raises(ValueError, match="shape"):
                ccr_mod.ccr_moe_experts_dgrad(c, [y], [w], ecnt, [x])
            with pytest.raises(ValueError, match="shape"):
                ccr_mod.ccr_moe_experts_wgrad(c, [x], [y], ecnt, [w])
            torch.cuda.synchronize()
            assert bool((w == 7.0).all()) and bool((y == 7.0).all()) and bool((x == 1.0).all())
        w = torch.ones(4, 16, H, **dev)
        ccr_mod.ccr_moe_experts(c, [x], [w], ecnt, [y])  # rows behind the last are left alone
        torch.cuda.synchronize()
    assert bool((y[:3] == H).all()) and bool((y[3:] == 7.0).all())
