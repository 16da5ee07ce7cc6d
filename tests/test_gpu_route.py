"""GPU parity of the router and its gradient with 64-bit references: choices are
equal, weights and gradients within their roundings."""
import pytest

from gpu_helpers import say, torch_cuda
from operator_helpers import Guarded, inside_nan

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NINF = float("-inf")


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


def scores_ref(l, score):
    import torch
    l = l.double()
    if score == "sigmoid":
        return torch.where(l == NINF, 0.0, 1 / (1 + torch.exp(-l)))
    m = l.max(1, keepdim=True).values
    z = torch.where(l == NINF, 0.0, torch.exp(l - torch.where(m == NINF, 0.0, m)))
    s = z.sum(1, keepdim=True)
    return torch.where(s == 0, 0.0, z / s)


def route_ref(l, bias, K, score, groups, kept, group_top, renorm, scale):
    """(topk, weights, scores) by sorting whole rows, on the CPU in 64 bits."""
    import torch
    l = l.cpu()
    T, E = l.shape
    s = scores_ref(l, score)
    open_ = l != NINF
    key = l.double() if bias is None else s + bias.cpu().double()
    if kept < groups:
        by = key if bias is not None or group_top == 1 else s
        by = torch.where(open_, by, NINF).view(T, groups, -1).nan_to_num(float("inf"), posinf=float("inf"), neginf=NINF)
        top = by.sort(dim=2, descending=True).values[:, :, :group_top]
        value = torch.where(top.isinf(), torch.where(top > 0, top, 0.0), top).sum(2)
        value = torch.where(top[:, :, 0] == NINF, NINF, value)
        best = value.sort(dim=1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros(T, groups, dtype=torch.bool).scatter(1, best, True)
        open_ = open_ & keep.repeat_interleave(E // groups, 1)
    # NaN above everything, closed experts behind everything
    order = torch.where(open_, key.nan_to_num(float("inf")), NINF).sort(dim=1, descending=True, stable=True).indices[:, :K]
    have = open_.gather(1, order)
    w = torch.where(have, s.gather(1, order), 0.0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    return torch.where(have, order, -1).int(), w * scale, s


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def run(ccr, ls, bs, K, how):
    import torch
    R, (T, E) = len(ls), ls[0].shape
    topk = [Guarded((T, K), torch.int32, fill=-9, offset_elements=1) for _ in ls]
    w = [Guarded((T, K), torch.float32, offset_elements=3) for _ in ls]
    counts = [Guarded((E,), torch.int64, fill=-9, offset_elements=1) for _ in ls]
    sums = [Guarded((E,), torch.float32, offset_elements=1) for _ in ls]
    work = Guarded((ccr.ccr_moe_route_work(R, T, E),), torch.float32)
    with ccr.Context(0) as c:
        ccr.ccr_moe_route(c, ls, [o.t for o in topk], [o.t for o in w], bias=bs, counts=[o.t for o in counts],
                          score_sums=[o.t for o in sums], work=work.t, **how)
        plain = [torch.empty(T, K, dtype=torch.int32, device="cuda") for _ in ls]
        pw = [torch.empty(T, K, device="cuda") for _ in ls]
        ccr.ccr_moe_route(c, ls, plain, pw, bias=bs, **how)
        torch.cuda.synchronize()
    assert all(o.intact() for o in (*topk, *w, *counts, *sums, work))
    for a, b, x, y in zip(topk, plain, w, pw):
        assert torch.equal(a.t, b) and torch.equal(x.t.nan_to_num(7.0), y.nan_to_num(7.0))
    return [[o.t for o in v] for v in (topk, w, counts, sums)]


def weight_units(score, E, K):
    """Roundings of a weight, in units U of it: the difference l - m carries half a
    unit of at most 64, the exponential two units, a softmax's sum a lane's 16 terms
    and six halvings of the wave, a sigmoid two operations; then the sum of the K,
    the quotient and the scale."""
    return (64 + 2 + 16 + 6 + 2 if score == "softmax" else 6) + K + 4 + 4


def check(ccr, ls, bs, K, how, what=""):
    import torch
    T, E = ls[0].shape
    say(f"route R={len(ls)} T={T} E={E} K={K} bias={bs is not None} {how} {what}")
    topk, w, counts, sums = run(ccr, ls, bs, K, how)
    units = weight_units(how["score"], E, K)
    for r, l in enumerate(ls):
        args = [how[k] for k in ("score", "groups", "kept", "group_top", "renorm", "scale")]
        wt, ww, s = route_ref(l, bs[r] if bs else None, K, *args)
        assert torch.equal(topk[r].cpu(), wt)
        assert bool(((w[r].cpu().double() - ww).abs() <= units * U * ww.abs() + 2.0 ** -140).all())
        assert torch.equal(counts[r].cpu(), torch.bincount(wt[wt >= 0].long().flatten(), minlength=E))
        # a slot's tokens one after the other, then fp64
        assert bool(((sums[r].cpu().double() - s.sum(0)).abs() <= (units + T + 8) * U * s.sum(0) + 2.0 ** -140).all())
    return topk, w


def how_(score="softmax", groups=1, kept=1, group_top=1, renorm=True, scale=1.0):
    return dict(score=score, groups=groups, kept=kept, group_top=group_top, renorm=renorm, scale=scale)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("R,T,E,K", [(1, 1, 1, 1), (1, 1, 64, 6), (2, 7, 3, 3), (1, 300, 60, 5), (3, 33, 64, 16),
                                     (1, 65, 65, 2), (1, 130, 256, 8), (2, 50, 255, 16), (1, 40, 257, 8),
                                     (1, 21, 1024, 16), (1, 9, 1000, 1), (64, 20, 8, 2), (1, 5000, 16, 4)])
def test_choices_and_weights(ccr_mod, R, T, E, K, score, with_bias):
    import torch
    g = gen(T * E + K)
    ls = [inside_nan(1.5 * torch.randn(T, E, generator=g, device="cuda"), 1) for _ in range(R)]
    bs = [inside_nan(0.1 * torch.randn(E, generator=g, device="cuda"), 1) for _ in range(R)] if with_bias else None
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        check(ccr_mod, ls, bs, K, how_(score, renorm=renorm, scale=scale))


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("T,E,K,groups,kept", [(1, 4, 2, 2, 1), (100, 64, 6, 8, 3), (64, 256, 8, 8, 4), (37, 60, 4, 4, 2),
                                               (20, 64, 3, 64, 5), (15, 1024, 16, 16, 4), (9, 320, 8, 5, 5),
                                               (50, 12, 2, 4, 3), (11, 1024, 8, 64, 1)])
def test_groups(ccr_mod, T, E, K, groups, kept, group_top, score, with_bias):
    import torch
    g = gen(T * E + groups)
    l = 1.5 * torch.randn(T, E, generator=g, device="cuda")
    bs = [0.1 * torch.randn(E, generator=g, device="cuda")] if with_bias else None
    check(ccr_mod, [l], bs, K, how_(score, groups, kept, group_top, scale=2.5))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(64, 1, 1), (256, 8, 4), (512, 1, 1)])
def test_keys_that_fp32_cannot_tell_apart(ccr_mod, E, groups, kept, score):
    """Biases that bring every key of a token to the same fp32 number: the choice is
    that of 64 bits."""
    import torch
    g = gen(E)
    l = torch.randn(1, E, generator=g, device="cuda").expand(30, E).contiguous()
    s = scores_ref(l[:1], score)[0]
    bias = (1.0 - s).float()
    assert (s.float() + bias).unique().numel() <= 3 < (s + bias.double()).unique().numel()
    for top in (1, 2):
        check(ccr_mod, [l], [bias], 8, how_(score, groups, kept, top))


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(64, 1, 1), (64, 8, 2), (256, 8, 4), (1024, 1, 1)])
def test_ties_go_to_the_lower_expert(ccr_mod, E, groups, kept, score, with_bias):
    import torch
    g = gen(E + groups)
    l = torch.randint(-2, 3, (200, E), generator=g, device="cuda").float()
    l[0] = 0.0
    l[1, ::2] = -0.0
    l[1, 1::2] = 0.0
    bs = [torch.zeros(E, device="cuda")] if with_bias else None
    topk, _ = check(ccr_mod, [l], bs, 6, how_(score, groups, kept, 2))
    assert topk[0][0].tolist() == list(range(6)) and topk[0][1].tolist() == list(range(6))


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,top", [(12, 1, 1, 1), (64, 8, 3, 2), (64, 8, 3, 1), (300, 4, 2, 2)])
def test_masked_experts_and_tokens(ccr_mod, E, groups, kept, top, score, with_bias):
    """Experts masked by -infinity are not chosen, whatever their bias; a token with
    fewer open experts than K ends in -1 with weight 0, one with none has no weight
    at all."""
    import torch
    g = gen(E)
    K, T = 4, 24
    l = torch.randn(T, E, generator=g, device="cuda")
    l[torch.rand(T, E, generator=g, device="cuda") < 0.5] = NINF
    l[0] = NINF
    l[1] = NINF
    l[1, E - 1] = 3.0
    l[2] = NINF
    l[2, [1, 2]] = torch.tensor([-80.0, 90.0], device="cuda")
    l[3] = -1e30
    bs = [10 * torch.rand(E, generator=g, device="cuda")] if with_bias else None
    topk, w = check(ccr_mod, [l], bs, K, how_(score, groups, kept, top))
    assert topk[0][0].tolist() == [-1] * K and not bool(w[0][0].any())
    assert topk[0][1].tolist() == [E - 1] + [-1] * (K - 1) and float(w[0][1, 0]) == 1.0


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score,group_top", [("softmax", 1), ("sigmoid", 2)])
@pytest.mark.parametrize("E,K,groups,kept", [(257, 4, 1, 1), (384, 8, 1, 1), (512, 16, 16, 5), (300, 7, 30, 6),
                                             (256, 8, 32, 8), (64, 3, 32, 2), (512, 8, 2, 1), (192, 8, 48, 10)])
def test_tokens_on_half_a_wave(ccr_mod, E, K, groups, kept, group_top, score, with_bias):
    import torch
    g = gen(E + groups)
    l = [1.5 * torch.randn(67, E, generator=g, device="cuda") for _ in range(2)]
    l[1][::3, 5] = NINF
    bs = [0.1 * torch.randn(E, generator=g, device="cuda")] * 2 if with_bias else None
    check(ccr_mod, l, bs, K, how_(score, groups, kept, group_top))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(64, 8, 2), (12, 4, 2), (256, 8, 3)])
def test_a_bias_of_minus_infinity_counts_in_its_group(ccr_mod, E, groups, kept, score):
    """The sum of a group's two largest keys is -infinity if the second one is, however
    near other groups are to each other; only masked logits are left out."""
    import torch
    g = gen(E + 5)
    T, K, eg = 40, 3, E // groups
    l = torch.randn(T, E, generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    bias[1:eg] = NINF                       # the first group: one key is not -infinity,
    bias[0] = 5.0                           # and it is the largest of all
    l[::2, -eg:] = l[::2, -2 * eg:-eg]      # two groups of the same value: decided in 64 bits
    bias[-eg:] = bias[-2 * eg:-eg]
    l[5, :eg] = NINF
    l[6, eg:] = NINF                        # the first group's value -infinity is above none at all
    topk = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_route(c, [l], [topk], [w], bias=[bias], score=score, groups=groups, kept=kept, group_top=2)
        torch.cuda.synchronize()
    keys = (scores_ref(l, score) + bias.double()).cpu()
    for t in range(T):
        open_ = [[e for e in range(i * eg, (i + 1) * eg) if float(l[t, e]) != NINF] for i in range(groups)]
        value = [sum(sorted((float(keys[t, e]) for e in o), reverse=True)[:2]) for o in open_]
        order = sorted((i for i in range(groups) if open_[i]), key=lambda i: (-value[i], i))[:kept]
        order += [i for i in range(groups) if not open_[i]][:kept - len(order)]
        chosen = sorted((e for i in order for e in open_[i]), key=lambda e: (-float(keys[t, e]), e))[:K]
        assert topk[t].tolist() == chosen + [-1] * (K - len(chosen)), t


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_shows_in_its_token_alone(ccr_mod, score):
    import torch
    l = torch.randn(6, 40, generator=gen(1), device="cuda")
    bad = l.clone()
    bad[2, 17] = float("nan")
    (t0,), (w0,) = run(ccr_mod, [l], None, 4, how_(score))[:2]
    (t1,), (w1,) = run(ccr_mod, [bad], None, 4, how_(score))[:2]
    rest = [0, 1, 3, 4, 5]
    assert torch.equal(t0[rest], t1[rest]) and torch.equal(w0[rest], w1[rest])
    assert 17 in t1[2].tolist() and bool(w1[2].isnan().all())
    assert bool(((t1 >= 0) & (t1 < 40)).all())


def test_same_choices_as_topk(ccr_mod):
    """Without bias and groups the choices are ccr_moe_topk's."""
    import torch
    l = torch.randn(500, 64, generator=gen(2), device="cuda")
    topk = torch.empty(500, 6, dtype=torch.int32, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_topk(c, l, topk)
        torch.cuda.synchronize()
    assert torch.equal(run(ccr_mod, [l], None, 6, how_())[0][0], topk)


# ------------------------------------------------------------------ backward
def backward_ref(l, topk, dw, dsum, score, renorm, scale):
    """(dlogits, the magnitude it is made of) in fp64, on the CPU."""
    import torch
    l, topk = l.cpu(), topk.cpu().long()
    s = scores_ref(l, score)
    E = l.shape[1]
    have = (topk >= 0) & (topk < E)
    at = torch.where(have, topk, 0)
    have = have & (l.gather(1, at) != NINF)
    c = torch.where(have, s.gather(1, at), 0.0)
    u = torch.where(have, dw.cpu().double() * scale, 0.0)
    mag = u.abs()
    if renorm:
        C = c.sum(1, keepdim=True)
        safe = torch.where(C == 0, 1.0, C)
        mag = torch.where(C == 0, 0.0, (mag + (mag * c).sum(1, keepdim=True) / safe) / safe)
        u = torch.where(C == 0, 0.0, (u - (u * c).sum(1, keepdim=True) / safe) / safe)
    ds = torch.zeros_like(s).scatter_add(1, at, torch.where(have, u, 0.0))
    dm = torch.zeros_like(s).scatter_add(1, at, torch.where(have, mag, 0.0))
    if dsum is not None:
        ds, dm = ds + dsum.cpu().double(), dm + dsum.cpu().double().abs()
    if score == "sigmoid":
        rest = 1 / (1 + torch.exp(l.double()))
        return s * rest * ds, s * rest * dm
    return s * (ds - (s * ds).sum(1, keepdim=True)), s * (dm + (s * dm).sum(1, keepdim=True))


def check_backward(ccr, ls, tops, dws, dsums, score, renorm, scale):
    import torch
    T, E = ls[0].shape
    K = tops[0].shape[1]
    say(f"route_bwd R={len(ls)} T={T} E={E} K={K} {score} renorm={renorm}")
    out = [Guarded((T, E), torch.float32, offset_elements=1) for _ in ls]
    with ccr.Context(0) as c:
        ccr.ccr_moe_route_bwd(c, ls, tops, dws, [o.t for o in out], dscore_sums=dsums, score=score, renorm=renorm,
                              scale=scale)
        torch.cuda.synchronize()
    # a score as a weight's, three times (in c, in C, in the last product); sums of
    # K, of a lane's 16 and six halvings
    units = 3 * weight_units(score, E, K) + 2 * K + 16 + 6 + 12
    for r, o in enumerate(out):
        assert o.intact()
        want, mag = backward_ref(ls[r], tops[r], dws[r], dsums[r] if dsums else None, score, renorm, scale)
        assert bool(((o.t.cpu().double() - want).abs() <= units * U * mag + 2.0 ** -140).all())
    return [o.t for o in out]


@pytest.mark.parametrize("with_sums", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("R,T,E,K", [(1, 1, 1, 1), (1, 1, 64, 6), (2, 7, 3, 3), (1, 300, 60, 5), (3, 33, 64, 16),
                                     (1, 130, 256, 8), (1, 40, 257, 8), (1, 21, 1024, 16), (64, 20, 8, 2)])
def test_backward(ccr_mod, R, T, E, K, score, renorm, with_sums):
    import torch
    g = gen(T + E)
    ls = [inside_nan(1.5 * torch.randn(T, E, generator=g, device="cuda"), 1) for _ in range(R)]
    tops = [torch.topk(l + torch.randn(T, E, generator=g, device="cuda"), K, dim=1).indices.int() for l in ls]
    dws = [inside_nan(torch.randn(T, K, generator=g, device="cuda"), 1) for _ in range(R)]
    dsums = [torch.randn(E, generator=g, device="cuda") for _ in range(R)] if with_sums else None
    check_backward(ccr_mod, ls, tops, dws, dsums, score, renorm, 2.5)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_of_absent_choices(ccr_mod, score, renorm):
    """Ids outside [0, E) and masked experts carry no gradient, their dweights (NaN
    here) are not used; an expert named twice collects both parts."""
    import torch
    g = gen(4)
    T, E, K = 12, 20, 4
    l, dw = torch.randn(T, E, generator=g, device="cuda"), torch.randn(T, K, generator=g, device="cuda")
    top = torch.topk(l, K, dim=1).indices.int()
    top[0, 1], top[1, 3], top[2, :], top[3, 0] = -1, E, -7, 2 ** 31 - 1
    l[4, top[4, 2].long()] = NINF
    l[5, 3:] = NINF
    top[5] = torch.tensor([0, 1, 2, 9], dtype=torch.int32)
    l[6] = NINF
    top[7, 3] = top[7, 0]
    l[8] = torch.linspace(-200, 90, E, device="cuda")
    top[8] = torch.tensor([0, 1, 2, 19], dtype=torch.int32)
    for t, k in ((0, 1), (1, 3), (2, 0), (3, 0), (4, 2), (5, 3), (6, 1)):
        dw[t, k] = float("nan")
    want = dw.clone().nan_to_num(0.0)
    ref = lambda d: backward_ref(l, top, d, None, score, renorm, 1.0)[0]
    (got,) = check_backward(ccr_mod, [l], [top], [want], None, score, renorm, 1.0)
    out = torch.empty(T, E, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_route_bwd(c, [l], [top], [dw], [out], score=score, renorm=renorm)
        torch.cuda.synchronize()
    assert torch.equal(out, got) and not bool(out[2].any()) and not bool(out[6].any())


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_against_differences(ccr_mod, score, renorm):
    """Central differences, in fp64, of <dw, weights> + <dsum, sums of scores> with
    the choices held: a step of 1e-3 leaves 1e-6 / 6 of a third derivative, below 50
    times the magnitude, and the fp32 gradient its roundings."""
    import torch
    g = gen(6)
    T, E, K, step = 3, 7, 3, 1e-3
    l, dw = torch.randn(T, E, generator=g, device="cuda"), torch.randn(T, K, generator=g, device="cuda")
    dsum = torch.randn(E, generator=g, device="cuda")
    top = torch.topk(l, K, dim=1).indices.int()
    out = torch.empty(T, E, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_route_bwd(c, [l], [top], [dw], [out], dscore_sums=[dsum], score=score, renorm=renorm, scale=2.0)
        torch.cuda.synchronize()

    def loss(x):
        s = scores_ref(x, score)
        w = s.gather(1, top.cpu().long())
        w = 2.0 * (w / w.sum(1, keepdim=True) if renorm else w)
        return (w * dw.cpu().double()).sum(1) + (s * dsum.cpu().double()).sum(1)

    mag = 4 * dw.abs().sum(1).cpu().double() + dsum.abs().sum().cpu().double()
    for e in range(E):
        d = torch.zeros(E, dtype=torch.float64)
        d[e] = step
        diff = (loss(l.cpu().double() + d) - loss(l.cpu().double() - d)) / (2 * step)
        assert bool(((out[:, e].cpu().double() - diff).abs() <= (50 * step ** 2 / 6 + 400 * U) * mag).all())


def test_streams_and_graph_replays(ccr_mod):
    import torch
    T, E, K = 700, 64, 6
    l, dw = torch.zeros(T, E, device="cuda"), torch.zeros(T, K, device="cuda")
    bias, dsum = torch.zeros(E, device="cuda"), torch.zeros(E, device="cuda")
    topk, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    counts, sums = torch.empty(E, dtype=torch.int64, device="cuda"), torch.empty(E, device="cuda")
    dl = torch.empty(T, E, device="cuda")
    work = [torch.empty(ccr_mod.ccr_moe_route_work(1, T, E), device="cuda") for _ in range(2)]
    outs = (topk, w, counts, sums, dl)
    with ccr_mod.Context(0) as c:
        def both(mine, stream=None):
            ccr_mod.ccr_moe_route(c, [l], [topk], [w], bias=[bias], score="sigmoid", groups=8, kept=3, group_top=2,
                                  counts=[counts], score_sums=[sums], work=work[mine], stream=stream)
            ccr_mod.ccr_moe_route_bwd(c, [l], [topk], [dw], [dl], dscore_sums=[dsum], score="sigmoid", stream=stream)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both(0)
        side = torch.cuda.Stream()
        for step in range(3):
            for t in (l, dw, bias, dsum):
                t.copy_(torch.randn(t.shape, device="cuda"))
            torch.cuda.synchronize()
            both(1, side)
            side.synchronize()
            want = [t.clone() for t in outs]
            for t in outs:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {step}"


def test_offsets_past_32_bits(ccr_mod):
    """Logits whose last row lies past 2^32 bytes from the first."""
    import torch
    T, E, K = 1100000, 1024, 2
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    say("route past 32-bit offsets")
    l = torch.zeros(T, E, device="cuda")
    l[-3:] = torch.randn(3, E, device="cuda")
    topk, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    dl, dw = torch.empty(T, E, device="cuda"), torch.ones(T, K, device="cuda")
    dw[:, 1] = 0.5
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_route(c, [l], [topk], [w])
        ccr_mod.ccr_moe_route_bwd(c, [l], [topk], [dw], [dl])
        torch.cuda.synchronize()
    want, ww, _ = route_ref(l[-3:], None, K, "softmax", 1, 1, 1, True, 1.0)
    assert torch.equal(topk[-3:].cpu(), want) and bool((topk[:-3] == torch.tensor([0, 1], device="cuda")).all())
    small = torch.empty(3, E, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_route_bwd(c, [l[-3:]], [topk[-3:]], [dw[-3:].contiguous()], [small])
        torch.cuda.synchronize()
    assert torch.equal(dl[-3:], small)


def test_empty_and_refusals(ccr_mod):
    import torch
    T, E, K = 5, 12, 3
    l = torch.randn(T, E, device="cuda")
    topk, w = torch.full((T, K), 7, dtype=torch.int32, device="cuda"), torch.full((T, K), 7.0, device="cuda")
    counts, sums = torch.full((E,), 7, dtype=torch.int64, device="cuda"), torch.full((E,), 7.0, device="cuda")
    dl = torch.full((T, E), 7.0, device="cuda")
    work = torch.empty(ccr_mod.ccr_moe_route_work(1, T, E), device="cuda")
    C = ccr_mod.CcrError
    with ccr_mod.Context(0) as c:
        route = lambda *a, **k: ccr_mod.ccr_moe_route(c, *a, **k)
        for args, kw, err, word in [
                (([l], [topk], [w]), dict(score="tanh"), ValueError, "score"),
                (([l], [topk], [w]), dict(groups=5), C, "groups"),
                (([l], [topk], [w]), dict(groups=0), C, "groups"),
                (([l], [topk], [w]), dict(groups=4, kept=5), C, "groups"),
                (([l], [topk], [w]), dict(groups=12, kept=2), C, "K = 3"),
                (([l], [topk], [w]), dict(groups=4, kept=2, group_top=3), C, "group_top"),
                (([l], [topk], [w]), dict(scale=float("inf")), C, "scale"),
                (([l], [topk], [w]), dict(counts=[counts]), ValueError, "work|shape|tensor"),
                (([l], [topk], [w]), dict(counts=[counts], work=work[:-1]), ValueError, "shape"),
                (([l], [topk], [w]), dict(counts=[counts.int()], work=work), TypeError, "counts"),
                (([l], [topk], [l.view(-1)[:T * K].view(T, K)]), {}, C, "overlap"),
                (([l], [topk.long()], [w]), {}, TypeError, "topk"),
                (([l.bfloat16()], [topk], [w]), {}, TypeError, "logits"),
                (([l[:, :2].contiguous()], [topk], [w]), {}, C, "K"),
                (([l], [topk], [w]), dict(bias=[sums[:-1]]), ValueError, "shape")]:
            with pytest.raises(err, match=word):
                route(*args, **kw)
        with pytest.raises(C, match="overlap"):
            ccr_mod.ccr_moe_route_bwd(c, [l], [topk], [w], [l])
        with pytest.raises(ValueError, match="shape"):
            ccr_mod.ccr_moe_route_bwd(c, [l], [topk], [w[:, :2].contiguous()], [dl])
        torch.cuda.synchronize()
        assert all(bool((t == 7).all()) for t in (topk, w, counts, sums, dl))
        ccr_mod.ccr_moe_route_bwd(c, [l[:0]], [topk[:0]], [w[:0]], [dl[:0]])
        route([l[:0]], [topk[:0]], [w[:0]], counts=[counts], score_sums=[sums])
        torch.cuda.synchronize()
    assert bool((topk == 7).all()) and not bool(counts.any()) and not bool(sums.any())
