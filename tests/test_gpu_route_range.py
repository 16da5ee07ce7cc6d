"""GPU parity of the router and its gradient with 64-bit references where fp32 is
short of range or of digits."""
import math

import pytest

from gpu_helpers import say, torch_cuda
from test_gpu_route import NINF, U, check, check_backward, gen, how_, weight_units

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


@pytest.mark.parametrize("size", [64.0, 1000.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,K", [(4, 2, 1, 2), (64, 8, 3, 6), (256, 8, 4, 8), (512, 16, 5, 8), (1024, 16, 4, 16)])
def test_groups_whose_two_keys_cancel(ccr_mod, E, groups, kept, K, score, size):
    """Biases of both signs: a group's value, the sum of its two best keys, is far
    smaller than they are, and what fp32 drops of the keys decides between groups
    of nearly the same value."""
    import torch
    g = gen(E + int(size))
    T, eg = 600, E // groups
    l = torch.randn(T, 1, eg, generator=g, device="cuda") + 1e-5 * torch.randn(T, groups, eg, generator=g, device="cuda")
    bias = torch.full((groups, eg), -size, device="cuda")
    bias[:, 0] = size
    check(ccr_mod, [l.view(T, E)], [bias.view(E)], K, how_(score, groups, kept, 2))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("kept", [5, 9, 15])
def test_groups_with_biases_of_every_size(ccr_mod, score, kept, top):
    """From 1e-30 to 3e38, and sums past fp32's range: every group twice, alike but
    for what is added to their logits."""
    import torch
    g = gen(top)
    T, E, groups = 300, 64, 16
    l = torch.randn(T, E, generator=g, device="cuda")
    l[:, 32:] = l[:, :32] + 1e-5 * torch.randn(T, 32, generator=g, device="cuda")
    size = torch.tensor([0.0, 1e-30, 0.1, 3.0, 1e4, 1e15, 3e38, 2.9e38], device="cuda")
    half = size[:, None] * torch.tensor([1.0, -1.0, -1.0, -1.0], device="cuda")
    half[-1] = 2.9e38
    half[0] = -2.9e38
    bias = torch.cat([half, half]).view(E)
    bias[:4] = -2.901e38
    check(ccr_mod, [l], [bias], 5, how_(score, groups, kept, top))


@pytest.mark.parametrize("with_sums", [False, True])
@pytest.mark.parametrize("E,K", [(3, 2), (64, 6), (200, 16), (300, 8), (1024, 16)])
def test_renormalised_gradient_of_tiny_scores(ccr_mod, E, K, with_sums):
    """Choices whose scores, or the quotients by their sum, are beyond fp32: sigmoids
    of logits down to -600, softmax choices as far below the largest logit."""
    import torch
    g = gen(E)
    below = torch.tensor([0.0, -40.0, -80.0, -88.0, -91.0, -95.0, -100.0, -104.0, -120.0, -300.0, -600.0], device="cuda")
    T = 3 * len(below)
    l = torch.randn(T, E, generator=g, device="cuda") + below.repeat(3)[:, None]
    l[-1, 1] = -30.0  # next to choices that vanish
    dw, dsum = torch.randn(T, K, generator=g, device="cuda"), torch.randn(E, generator=g, device="cuda")
    top = (1 + torch.argsort(torch.rand(T, E - 1, generator=g, device="cuda"), dim=1)[:, :K]).int()
    top[-1, 0] = 1
    dsums = [dsum] if with_sums else None
    check_backward(ccr_mod, [l], [top], [dw], dsums, "sigmoid", True, 2.5)
    l[:, 0] = 1.0  # in no choice
    check_backward(ccr_mod, [l], [top], [dw], dsums, "softmax", True, 2.5)


@pytest.mark.parametrize("E,K", [(3, 2), (64, 6), (200, 16), (300, 8), (1024, 16)])
def test_renormalised_weights_of_tiny_scores(ccr_mod, E, K):
    """Weights of choices whose scores are below fp32's normal numbers are those of 64
    bits: sigmoids of logits down to -600, and 0 at -800; softmax choices as far
    below an expert that the bias keeps out."""
    import torch
    g = gen(E)
    below = torch.tensor([0.0, -40.0, -80.0, -88.0, -91.0, -95.0, -100.0, -104.0, -120.0, -300.0, -600.0, -800.0],
                         device="cuda")
    T = 3 * len(below)
    l = torch.randn(T, E, generator=g, device="cuda") + below.repeat(3)[:, None]
    l[5, 1] = -30.0  # next to choices that vanish
    check(ccr_mod, [l], None, K, how_("sigmoid"))
    l[:, 0] = 1.0
    bias = torch.zeros(E, device="cuda")
    bias[0] = -10.0
    check(ccr_mod, [l], [bias], K, how_("softmax", scale=2.5))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [12, 256, 1024])
def test_tokens_with_tiny_scores_leave_others_alone(ccr_mod, E, score):
    """A token's results do not hang on the tokens beside it: infinities and NaN that
    the bias keeps out of the choices, scores around 2^-126 and ordinary ones."""
    import torch
    K, g = 3, gen(E)
    l = torch.randn(40, E, generator=g, device="cuda")
    l[:, 4:] -= torch.linspace(0, 100, 40, device="cuda")[:, None]
    l[3, 0], l[8, 1], l[13, 2] = float("inf"), float("nan"), NINF
    bias = torch.zeros(E, device="cuda")
    bias[:4] = -10.0
    far = l.clone()
    far[::2, 4:] = -200.0
    far[::2, :4] = 0.0
    out = []
    with ccr_mod.Context(0) as c:
        for v in (l, far):
            topk, w = torch.empty(40, K, dtype=torch.int32, device="cuda"), torch.empty(40, K, device="cuda")
            dl, dw = torch.empty(40, E, device="cuda"), torch.ones(40, K, device="cuda")
            dw[:, 1] = 0.5
            ccr_mod.ccr_moe_route(c, [v], [topk], [w], bias=[bias], score=score)
            ccr_mod.ccr_moe_route_bwd(c, [v], [topk], [dw], [dl], score=score)
            torch.cuda.synchronize()
            out.append([t[1::2].nan_to_num(7.0) for t in (topk, w, dl)])
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("E,chain", [(64, 1024), (256, 1024), (512, 2048), (1024, 4096)])
def test_sums_of_scores_over_many_tokens(ccr_mod, E, chain):
    """Every token the same score, 0.49 units above a multiple of what a sum of `chain`
    of them resolves, so that it would drift apart from the true one: chains of at
    most 128 additions each."""
    import torch
    R, T = 64, 262143
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB")
    say(f"route sums over {R} x {T} tokens E={E}")
    unit = 2.0 ** (math.floor(math.log2(0.24 * chain)) - 23)
    score = (math.floor(0.24 / unit) + 0.49) * unit
    l = torch.full((T, E), math.log(score / (1 - score)), device="cuda")
    topk = [torch.empty(T, 1, dtype=torch.int32, device="cuda") for _ in range(R)]
    w = [torch.empty(T, 1, device="cuda") for _ in range(R)]
    counts = [torch.empty(E, dtype=torch.int64, device="cuda") for _ in range(R)]
    sums = [torch.empty(E, device="cuda") for _ in range(R)]
    work = torch.empty(ccr_mod.ccr_moe_route_work(R, T, E), device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_route(c, [l] * R, topk, w, score="sigmoid", counts=counts, score_sums=sums, work=work)
        torch.cuda.synchronize()
    want = T / (1 + math.exp(-float(l[0, 0])))
    # 128 tokens to a lane, the lanes of four waves; then fp64, and its rounding
    units = weight_units("sigmoid", E, 1) + 128 + 16 + 1
    worst = max(float((v.double() - want).abs().max()) for v in sums) / (U * want)
    assert worst <= units, f"{worst} units"
    for r in range(R):
        assert counts[r].tolist() == [T] + [0] * (E - 1)
