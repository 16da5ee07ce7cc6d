"""GPU parity of the gated sum and its gradients with a 64-bit reference."""
import pytest

from gpu_helpers import say, torch_cuda
from operator_helpers import Guarded, HALF, inside_nan, tdtype

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a unit of an fp32 value, relative


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


def reference(rows, logits, topk, norm, dy=None):
    """fp64: (w, y) or (w, drows, dlogits, magnitude of each dlogit)."""
    import torch
    T, K, H = rows.shape
    E = logits.shape[1]
    l = logits.double()
    have = (topk >= 0) & (topk < E)
    at = torch.where(have, topk, 0).long()
    lk = torch.where(have, l.gather(1, at), float("-inf"))
    have = have & (lk != float("-inf"))
    base = l if norm == "all" else torch.where(have, lk, float("-inf"))
    m = base.max(dim=1, keepdim=True).values
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    z = torch.exp(base - m).sum(dim=1, keepdim=True)
    w = torch.where(have, torch.exp(lk - m) / z, 0.0)
    x = torch.where(have[:, :, None], rows.double(), 0.0)
    if dy is None:
        return w, (w[:, :, None] * x).sum(1), (w[:, :, None] * x.abs()).sum(1)
    d = dy.double()
    g = (x * d[:, None, :]).sum(2)
    G = (x.abs() * d.abs()[:, None, :]).sum(2)
    s, S = (w * g).sum(1, keepdim=True), (w * G).sum(1, keepdim=True)
    drows = torch.where(have[:, :, None], w[:, :, None] * d[:, None, :], 0.0)
    dl, mag = torch.zeros_like(l), torch.zeros_like(l)
    if norm == "all":
        p = torch.where(z > 0, torch.exp(l - m) / z, 0.0)
        dl, mag = dl - p * s, mag + p * S
        part, pmag = w * g, w * G
    else:
        part, pmag = w * (g - s), w * (G + S)
    dl = dl.scatter_add(1, at, torch.where(have, part, 0.0))
    mag = mag.scatter_add(1, at, torch.where(have, pmag, 0.0))
    return w, drows, dl, mag


def inputs(T, E, K, H, dt, seed, offset=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    rows = inside_nan(rnd(T, K, H).to(tdtype(dt)))
    logits = inside_nan(1.5 * rnd(T, E))
    topk = torch.topk(logits, K, dim=1).indices.to(torch.int32)
    dy = inside_nan(rnd(T, H).to(tdtype(dt)))
    return rows, logits, topk, dy


def check(ccr, sets, norm, dt):
    import torch
    R = len(sets)
    T, K, H = sets[0][0].shape
    E = sets[0][1].shape[1]
    say(f"gate R={R} T={T} E={E} K={K} H={H} {dt} {norm}")
    rows, logits, topk, dy = (list(x) for x in zip(*sets))
    y = [Guarded((T, H), tdtype(dt)) for _ in sets]
    dr = [Guarded((T, K, H), tdtype(dt)) for _ in sets]
    dl = [Guarded((T, E), torch.float32) for _ in sets]
    with ccr.Context(0) as c:
        ccr.ccr_moe_gate_sum(c, rows, logits, topk, [o.t for o in y], norm=norm)
        ccr.ccr_moe_gate_sum_bwd(c, dy, rows, logits, topk, [o.t for o in dr], [o.t for o in dl], norm=norm)
        torch.cuda.synchronize()
    # A weight: the difference l - m carries half a unit of at most |l - m| < 64,
    # the exponential 2 units, the sum up to n terms as many each, the quotient
    # one: below (64 + n + 8) units of the weight in all, n = K or E / 64 + 6
    # additions (a lane's terms one by one, then six halvings of the wave).
    n = 64 + 8 + (K if norm == "chosen" else E // 64 + 7)
    for r in range(R):
        assert y[r].intact() and dr[r].intact() and dl[r].intact()
        w, want, mag = reference(rows[r], logits[r], topk[r], norm)
        got = y[r].t.double()
        assert bool(((got - want).abs() <= HALF[dt] * want.abs() + (n + K + 1) * U * mag * 1.01).all())
        w, wdr, wdl, dmag = reference(rows[r], logits[r], topk[r], norm, dy[r])
        err = (dr[r].t.double() - wdr).abs()
        assert bool((err <= (HALF[dt] + (n + 1) * U) * 1.01 * wdr.abs()).all())
        # g_k sums H products, s the K of them; both are then weighted
        tol = (2 * n + H + K + 4) * U * 1.01 * dmag
        assert bool(((dl[r].t.double() - wdl).abs() <= tol).all())
    return y, dr, dl


@pytest.mark.parametrize("norm", ["chosen", "all"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,K,H", [(1, 4, 1, 8), (1, 64, 6, 2048), (7, 8, 8, 24), (130, 60, 3, 512),
                                     (33, 1024, 16, 136), (5, 16, 2, 4104), (64, 3, 3, 1032), (300, 64, 5, 520)])
def test_against_the_reference(ccr_mod, T, E, K, H, dt, norm):
    check(ccr_mod, [inputs(T, E, K, H, dt, T + E)], norm, dt)


def test_several_ranks(ccr_mod):
    check(ccr_mod, [inputs(37, 16, 4, 264, "bf16", s) for s in range(5)], "chosen", "bf16")


@pytest.mark.parametrize("norm", ["chosen", "all"])
@pytest.mark.parametrize("H", [256, 4096])
def test_absent_choices_are_not_read(ccr_mod, norm, H):
    """Dropped choices (ids outside [0, E)) and masked experts (logit -inf):
    weight 0, their rows -- NaN and infinities here -- not read; a token
    without any choice gets zeros."""
    import torch
    T, E, K = 24, 12, 4
    rows, logits, topk, dy = inputs(T, E, K, H, "bf16", 3)
    topk[0, 1] = -1
    topk[1, 3] = E
    topk[2, :] = -7
    topk[3, 0] = 2 ** 31 - 1
    for t, k in [(4, 0), (5, 3)]:
        logits[t, topk[t, k].long()] = float("-inf")
    logits[6, :] = float("-inf")
    logits[7, topk[7, 1:].long()] = float("-inf")
    for t, k in [(0, 1), (1, 3), (2, 0), (2, 2), (3, 0), (4, 0), (5, 3), (6, 0), (7, 2)]:
        rows[t, k] = float("nan") if (t + k) % 2 else float("inf")
    y, dr, dl = check(ccr_mod, [(rows, logits, topk, dy)], norm, "bf16")
    for t in (2, 6):
        assert bool((y[0].t[t] == 0).all()) and bool((dr[0].t[t] == 0).all()) and bool((dl[0].t[t] == 0).all())
    assert torch.equal(y[0].t[7], rows[7, 0]) or norm == "all"


@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_the_same_expert_twice_and_large_logits(ccr_mod, norm):
    rows, logits, topk, dy = inputs(20, 8, 3, 64, "f32", 5)
    topk[:, 2] = topk[:, 0]
    logits[3] *= 20
    logits[4] += 2.0 ** 12
    check(ccr_mod, [(rows, logits, topk, dy)], norm, "f32")


def test_nan_logit_makes_its_token_nan(ccr_mod):
    import torch
    rows, logits, topk, dy = inputs(6, 8, 2, 32, "f32", 6)
    logits[2, topk[2, 0].long()] = float("nan")
    y = torch.zeros(6, 32, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_gate_sum(c, [rows], [logits], [topk], [y])
        torch.cuda.synchronize()
    assert bool(y[2].isnan().all()) and not bool(y[[0, 1, 3, 4, 5]].isnan().any())


@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_dlogits_against_differences(ccr_mod, norm):
    """Central differences of <dy, y> in fp64: step h leaves h^2 / 6 times a
    third derivative, bounded by 13 times the sum of the weighted magnitudes
    (each derivative of a softmax weight is at most a few times the weight),
    and the fp32 gradient its own rounding."""
    import torch
    T, E, K, H = 4, 6, 3, 16
    rows, logits, topk, dy = inputs(T, E, K, H, "f32", 8)
    dr, dl = torch.empty(T, K, H, device="cuda"), torch.empty(T, E, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_gate_sum_bwd(c, [dy], [rows], [logits], [topk], [dr], [dl], norm=norm)
        torch.cuda.synchronize()
    step = 1e-3
    _, _, scale = reference(rows, logits, topk, norm)
    G = (scale * dy.double().abs()).sum(1)
    for e in range(E):
        up, down = logits.double().clone(), logits.double().clone()
        up[:, e] += step
        down[:, e] -= step
        f = lambda l: (reference(rows, l, topk, norm)[1] * dy.double()).sum(1)
        diff = (f(up) - f(down)) / (2 * step)
        assert bool(((dl[:, e].double() - diff).abs() <= (13 * step ** 2 / 6 + 400 * U) * G).all())


def test_streams_and_graph_replays(ccr_mod):
    import torch
    T, E, K, H = 50, 16, 4, 520
    rows, logits, topk, dy = inputs(T, E, K, H, "bf16", 9)
    y, dr, dl = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty_like(rows),
                 torch.empty_like(logits))
    with ccr_mod.Context(0) as c:
        def both(stream=None):
            ccr_mod.ccr_moe_gate_sum(c, [rows], [logits], [topk], [y], stream=stream)
            ccr_mod.ccr_moe_gate_sum_bwd(c, [dy], [rows], [logits], [topk], [dr], [dl], stream=stream)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
        side = torch.cuda.Stream()
        for step in range(3):
            rows.copy_(torch.randn(T, K, H, device="cuda").to(torch.bfloat16))
            logits.copy_(torch.randn(T, E, device="cuda"))
            torch.cuda.synchronize()
            both(side)
            side.synchronize()
            want = [t.clone() for t in (y, dr, dl)]
            for t in (y, dr, dl):
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((y, dr, dl), want)), f"replay {step}"


def test_offsets_past_32_bits(ccr_mod):
    """The last tokens' rows lie past 2^32 bytes from the first."""
    import torch
    T, E, K, H = 70000, 8, 4, 8192
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    say("gate past 32-bit offsets")
    rows = torch.zeros(T, K, H, dtype=torch.bfloat16, device="cuda")
    rows[-3:] = torch.randn(3, K, H, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, device="cuda")
    topk = torch.topk(logits, K, dim=1).indices.to(torch.int32)
    dy = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    dr, dl = torch.empty_like(rows), torch.empty_like(logits)
    small = [t[-3:].contiguous() for t in (rows, logits, topk, dy)]
    sy, sdr, sdl = (torch.empty_like(t) for t in (small[3], small[0], small[1]))
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_gate_sum(c, [rows], [logits], [topk], [y])
        ccr_mod.ccr_moe_gate_sum_bwd(c, [dy], [rows], [logits], [topk], [dr], [dl])
        ccr_mod.ccr_moe_gate_sum(c, [small[0]], [small[1]], [small[2]], [sy])
        ccr_mod.ccr_moe_gate_sum_bwd(c, [small[3]], [small[0]], [small[1]], [small[2]], [sdr], [sdl])
        torch.cuda.synchronize()
    assert torch.equal(y[-3:], sy) and torch.equal(dr[-3:], sdr) and torch.equal(dl[-3:], sdl)
    assert not bool(y[:-3].any()) and not bool(dl[:-3].any())


def test_empty_and_refusals(ccr_mod):
    import torch
    rows, logits, topk, dy = inputs(4, 8, 2, 16, "bf16", 1)
    y = torch.full((4, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_gate_sum(c, [rows[:0]], [logits[:0]], [topk[:0]], [y[:0]])
        with pytest.raises(ccr_mod.CcrError, match="overlap"):
            ccr_mod.ccr_moe_gate_sum(c, [rows], [logits], [topk], [rows.view(-1)[:64].view(4, 16)])
        with pytest.raises(ccr_mod.CcrError, match="16 bytes"):
            ccr_mod.ccr_moe_gate_sum(c, [rows[:, :, :4].contiguous()], [logits], [topk],
                                     [y[:, :4].contiguous()])
        with pytest.raises(ValueError):
            ccr_mod.ccr_moe_gate_sum(c, [rows], [logits], [topk], [y], norm="none")
        with pytest.raises(TypeError):
            ccr_mod.ccr_moe_gate_sum(c, [rows], [logits], [topk.long()], [y])
        with pytest.raises(ccr_mod.CcrError, match="K"):
            ccr_mod.ccr_moe_gate_sum(c, [rows], [logits[:, :1].contiguous()], [topk], [y])
        torch.cuda.synchronize()
    assert bool((y == 7.0).all())
