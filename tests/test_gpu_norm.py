"""GPU parity of the root-mean-square norm with residual, its 8-bit rows and its
gradients with 64-bit references."""
import numpy as np
import pytest

import rows8_helpers as r8
from gpu_helpers import say, torch_cuda
from operator_helpers import Guarded, HALF, inside_nan, tdtype

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a unit of an fp32 value, relative
EPS = 1e-5


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


def rnd(g, *shape):
    import torch
    return torch.randn(shape, generator=g, device="cuda")


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def forward_ref(x, res, w, eps=EPS):
    """(h in its type, rstd, y) in fp64."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hd = h.double()
    rstd = (hd.square().mean(dim=1) + eps).rsqrt()
    return h, rstd, hd * rstd[:, None] * w.double()


def check_q8(rows, y, rel):
    """Packed rows against y (fp64, known to `rel`): every value within half a step
    of e4m3 (2^-4 of it, or 2^-10 of the scale among the smallest), the scale the
    smallest that holds the block, zeros behind."""
    rows, y = rows.cpu().numpy(), y.cpu().numpy()
    H = y.shape[1]
    V = -(-H // 128) * 128
    v, s = r8.unpack(rows, H)
    assert not rows[:, H:V].any() and not rows[:, V + V // 32:].any()
    full = np.zeros((len(y), V))
    full[:, :H] = y
    top = np.abs(full).reshape(len(y), -1, 32).max(axis=2)
    scale = np.ldexp(1.0, s - 127)
    assert (448 * scale >= top * (1 - rel)).all()
    assert ((224 * scale < top * (1 + rel)) | (s == 0)).all()
    step = np.repeat(scale, 32, axis=1)[:, :H]
    assert (np.abs(v - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * step) * (1 + rel) + rel * np.abs(y)).all()


def check(ccr, R, T, H, dt, wdt, add, seed, make=None):
    import torch
    say(f"norm R={R} T={T} H={H} {dt} w {wdt} add={add}")
    g = gen(seed)
    d = tdtype(dt)
    xs = [rnd(g, T, H).to(d) for _ in range(R)]
    rs = [(3 * rnd(g, T, H)).to(d) for _ in range(R)] if add else None
    if make:
        make(xs, rs)
    xs = [inside_nan(x) for x in xs]
    rs = [inside_nan(x) for x in rs] if add else None
    ws = [inside_nan((1 + 0.2 * rnd(g, H)).to(tdtype(wdt))) for _ in range(R)]
    y = [Guarded((T, H), d) for _ in range(R)]
    q = [Guarded((T, r8.row_bytes(H)), torch.uint8, fill=7) for _ in range(R)]
    h = [Guarded((T, H), d) for _ in range(R)] if add else None
    rstd = [Guarded((T,), torch.float32, offset_elements=1) for _ in range(R)]
    more = dict(residual=rs, h=[o.t for o in h]) if add else {}
    with ccr.Context(0) as c:
        ccr.ccr_rms_norm(c, xs, ws, y=[o.t for o in y], q=[o.t for o in q], rstd=[o.t for o in rstd], eps=EPS, **more)
        only = [torch.empty(T, H, dtype=d, device="cuda") for _ in range(R)]
        ccr.ccr_rms_norm(c, xs, ws, y=only, eps=EPS, **more)
        only8 = [torch.full((T, r8.row_bytes(H)), 7, dtype=torch.uint8, device="cuda") for _ in range(R)]
        ccr.ccr_rms_norm(c, xs, ws, q=only8, eps=EPS, **more)
        torch.cuda.synchronize()
    for r in range(R):
        wh, wr, wy = forward_ref(xs[r], rs[r] if add else None, ws[r])
        assert all(o[r].intact() for o in (y, q, rstd)) and (not add or h[r].intact())
        if add:
            assert torch.equal(h[r].t, wh)
        # rstd is rounded once from 64 bits; y takes two more products
        assert bool(((rstd[r].t.double() - wr).abs() <= 1.01 * U * wr).all())
        # (below the smallest normal number each of three roundings is off by half
        # the smallest step)
        least = 2.0 ** -149 * 3 + (2.0 ** -134 if dt == "bf16" else 0)
        assert bool(((y[r].t.double() - wy).abs() <= (HALF[dt] + 3.1 * U) * wy.abs() + least).all())
        check_q8(q[r].t, wy, 3.1 * U)
        assert torch.equal(only[r], y[r].t) and torch.equal(only8[r], q[r].t)


SHAPES = [(1, 1, 8), (1, 1, 2048), (3, 5, 24), (2, 7, 520), (1, 3, 4104), (1, 2, 16392), (1, 70, 1032),
          (2, 300, 64), (1, 9, 128), (1, 2, 8200)]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("R,T,H", SHAPES + [(1, 4, 20)])
def test_forward(ccr_mod, R, T, H, dt, wdt, add):
    if H % 8 and dt == "bf16":
        pytest.skip("no whole vectors")
    check(ccr_mod, R, T, H, dt, wdt, add, T + H)


def test_extreme_rows(ccr_mod):
    """Zeros, values whose squares overflow or vanish in fp32, one large value."""
    import torch

    def make(xs, rs):
        xs[0][0] = 0
        xs[0][1] *= 1e30
        xs[0][2] *= 1e-30
        xs[0][3, 5] = 3e38
        xs[0][4] = 0
        xs[0][4, 7] = 1e-40

    check(ccr_mod, 1, 6, 264, "f32", "f32", False, 3, make)
    check(ccr_mod, 1, 6, 264, "bf16", "bf16", False, 4, make)


def test_not_finite_rows_stay_apart(ccr_mod):
    """A row with an infinity has rstd 0, one with a NaN is NaN; 8-bit blocks with
    either stand for NaN; the other rows are as without them."""
    import torch
    T, H = 5, 160
    x = rnd(gen(1), T, H)
    w = torch.ones(H, device="cuda")
    bad = x.clone()
    bad[1, 40] = float("inf")
    bad[3, 100] = float("nan")
    out = []
    with ccr_mod.Context(0) as c:
        for v in (x, bad):
            y, rstd = torch.empty(T, H, device="cuda"), torch.empty(T, device="cuda")
            q = torch.empty(T, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
            back = torch.empty(T, H, device="cuda")
            ccr_mod.ccr_rms_norm(c, [v], [w], y=[y], q=[q], rstd=[rstd])
            ccr_mod.ccr_dequantize_rows(c, [q], [back])
            torch.cuda.synchronize()
            out.append((y, rstd, back))
    (y0, r0, b0), (y1, r1, b1) = out
    keep = [0, 2, 4]
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(b0[keep], b1[keep]) and torch.equal(r0[keep], r1[keep])
    assert float(r1[1]) == 0 and bool(y1[1, 40].isnan()) and not bool(y1[1, :40].any()) and not bool(y1[1, 41:].any())
    assert bool(b1[1, 32:64].isnan().all()) and not bool(b1[1, :32].any()) and not bool(b1[1, 64:].any())
    assert bool(r1[3].isnan()) and bool(y1[3].isnan().all()) and bool(b1[3].isnan().all())


@pytest.mark.parametrize("H", [64, 2048, 16392])
def test_h_in_the_place_of_x_or_of_the_residual(ccr_mod, H):
    import torch
    g = gen(H)
    x, res = rnd(g, 6, H).bfloat16(), rnd(g, 6, H).bfloat16()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    want_h, want_y, y = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_rms_norm(c, [x], [w], y=[want_y], residual=[res], h=[want_h])
        for into in (0, 1):
            a = [x.clone(), res.clone()]
            y.zero_()
            ccr_mod.ccr_rms_norm(c, [a[0]], [w], y=[y], residual=[a[1]], h=[a[into]])
            torch.cuda.synchronize()
            assert torch.equal(a[into], want_h) and torch.equal(y, want_y)
            assert torch.equal(a[1 - into], (x, res)[1 - into])


def backward_ref(dy, h, w, rstd, dh):
    """(dx, dw, and the sums of the magnitudes that each is made of) in fp64."""
    d, r = dy.double(), rstd.double()[:, None]
    hh, gg = h.double() * r, d * w.double()
    s, S = (gg * hh).mean(1, keepdim=True), (gg * hh).abs().mean(1, keepdim=True)
    dx, mag = r * (gg - hh * s), r * (gg.abs() + hh.abs() * S)
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    return dx, (d * hh).sum(0), mag, (d * hh).abs().sum(0)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("R,T,H", SHAPES + [(1, 1500, 264), (64, 20, 40)])
def test_backward(ccr_mod, R, T, H, dt, wdt, add):
    import torch
    ccr = ccr_mod
    say(f"norm_bwd R={R} T={T} H={H} {dt} w {wdt} add={add}")
    g = gen(T * H)
    d = tdtype(dt)
    dy, h = ([inside_nan((k * rnd(g, T, H)).to(d)) for _ in range(R)] for k in (1, 2))
    dh = [inside_nan(rnd(g, T, H).to(d)) for _ in range(R)] if add else None
    w = [inside_nan((1 + 0.2 * rnd(g, H)).to(tdtype(wdt))) for _ in range(R)]
    rstd = [inside_nan((x.double().square().mean(1) + EPS).rsqrt().float(), 1) for x in h]
    dx = [Guarded((T, H), d) for _ in range(R)]
    dw = [Guarded((H,), torch.float32, offset_elements=1) for _ in range(R)]
    n = ccr.ccr_rms_norm_work(R, T, H)
    work = Guarded((n,), torch.float32)
    with ccr.Context(0) as c:
        ccr.ccr_rms_norm_bwd(c, dy, h, w, rstd, [o.t for o in dx], [o.t for o in dw], work.t, dh=dh)
        torch.cuda.synchronize()
        first = [o.t.clone() for o in dw]
        work.t.fill_(float("nan"))
        ccr.ccr_rms_norm_bwd(c, dy, h, w, rstd, [o.t for o in dx], [o.t for o in dw], work.t, dh=dh, accumulate=True)
        torch.cuda.synchronize()
    assert work.intact()
    for r in range(R):
        assert dx[r].intact() and dw[r].intact()
        wdx, wdw, mag, wmag = backward_ref(dy[r], h[r], w[r], rstd[r], dh[r] if add else None)
        # the row's sum: a lane adds at most 32 values, or H / 256 of a longer row,
        # then ten sums of lanes and waves; a dozen products on the way
        n = 32 + H // 256 + 10 + 12
        assert bool(((dx[r].t.double() - wdx).abs() <= HALF[dt] * wdx.abs() + n * U * mag).all())
        assert bool(((first[r].double() - wdw).abs() <= (T + 16) * U * wmag).all())
        assert torch.equal(dw[r].t, first[r] + first[r])  # the same sum, added to the first


def test_backward_against_differences(ccr_mod):
    """Central differences of <dy, y> + <dh, h> in fp64, of step e: off by e^2 / 6 of
    a third derivative, below 100 times the sum of the magnitudes (values around
    1, H = 12), and the fp32 gradient by its own roundings."""
    import torch
    T, H, step = 3, 12, 1e-3
    g = gen(5)
    h, dy, dh, w = rnd(g, T, H), rnd(g, T, H), rnd(g, T, H), 1 + 0.2 * rnd(g, H)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx, dw = torch.empty(T, H, device="cuda"), torch.empty(H, device="cuda")
    work = torch.empty(ccr_mod.ccr_rms_norm_work(1, T, H), device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_rms_norm_bwd(c, [dy], [h], [w], [rstd], [dx], [dw], work, dh=[dh])
        torch.cuda.synchronize()

    def loss(hh, ww):
        r = (hh.square().mean(1, keepdim=True) + EPS).rsqrt()
        return ((hh * r * ww * dy.double()) + hh * dh.double()).sum(1)

    mag = (dy.abs() * w.abs()).sum(1).double() + dh.abs().sum(1).double()
    for i in range(H):
        e = torch.zeros(H, dtype=torch.float64, device="cuda")
        e[i] = step
        diff = (loss(h.double() + e, w.double()) - loss(h.double() - e, w.double())) / (2 * step)
        assert bool(((dx[:, i].double() - diff).abs() <= (100 * step ** 2 / 6 + 100 * U) * mag).all())
        diff = (loss(h.double(), w.double() + e) - loss(h.double(), w.double() - e)).sum() / (2 * step)
        assert abs(float(dw[i]) - float(diff)) <= 100 * U * float(mag.sum()) + 1e-9


@pytest.mark.parametrize("H", [32, 64, 2048, 16392])
def test_roots_over_the_whole_range(ccr_mod, H):
    """rstd of rows of every magnitude of fp32, of zeros and of infinities, without an
    eps, and of one: off by its rounding to fp32 and 2^-40 before."""
    import torch
    sizes = [0.0, 1.4e-45, 1e-38, 3e-20, 1.0, 7e19, 3.4e38, float("inf")]
    x = torch.tensor(sizes, device="cuda")[:, None] * torch.ones(H, device="cuda")
    x[3:6] *= 0.5 + torch.rand(3, H, generator=gen(H), device="cuda")
    w, y, rstd = torch.ones(H, device="cuda"), torch.empty_like(x), torch.empty(len(sizes), device="cuda")
    with ccr_mod.Context(0) as c:
        for eps in (0.0, 1e-6):
            ccr_mod.ccr_rms_norm(c, [x], [w], y=[y], rstd=[rstd], eps=eps)
            torch.cuda.synchronize()
            want = 1.0 / (x.double().square().mean(1) + float(torch.tensor(eps))).sqrt()
            big = want > torch.finfo(torch.float32).max  # infinite in fp32
            got = rstd.double()
            assert bool((got[big] == float("inf")).all())
            # 1 / 3.4e38 = 2.9e-39 lies below 2^-126 = 1.2e-38, where fp32's steps are all
            # 2^-149 and half a step is 2^-150
            assert bool(((got - want).abs() <= want * U * (1 + 2.0 ** -15) + 2.0 ** -150)[~big].all())


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dt,wdt", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("R,T,H", [(3, 37, 56), (2, 50, 200), (2, 41, 384), (1, 33, 960), (1, 19, 2040), (1, 6, 16384)])
def test_rows_of_every_length(ccr_mod, R, T, H, dt, wdt, add):
    """Numbers of rows that end inside a wave and a workgroup, in rows of sixteenths of
    a wave's lanes up to several vectors to each lane of a workgroup."""
    test_forward(ccr_mod, R, T, H, dt, wdt, add)
    test_backward(ccr_mod, R, T, H, dt, wdt, add)


@pytest.mark.parametrize("H", [64, 2048, 16392])
def test_dx_in_the_place_of_dh(ccr_mod, H):
    import torch
    g = gen(H)
    T = 5
    h, dy, dh = (rnd(g, T, H).bfloat16() for _ in range(3))
    w = torch.ones(H, device="cuda")
    rstd = torch.ones(T, device="cuda")
    dx, dw, dw2 = torch.empty_like(h), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    work = torch.empty(ccr_mod.ccr_rms_norm_work(1, T, H), device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_rms_norm_bwd(c, [dy], [h], [w], [rstd], [dx], [dw], work, dh=[dh])
        ccr_mod.ccr_rms_norm_bwd(c, [dy], [h], [w], [rstd], [dh], [dw2], work, dh=[dh])
        torch.cuda.synchronize()
    assert torch.equal(dh, dx) and torch.equal(dw, dw2)


def test_streams_and_graph_replays(ccr_mod):
    import torch
    T, H = 40, 520
    x, res, dy, dh = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    h, y, dx = (torch.empty_like(x) for _ in range(3))
    q = torch.empty(T, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    rstd, dw = torch.empty(T, device="cuda"), torch.empty(H, device="cuda")
    work = [torch.empty(ccr_mod.ccr_rms_norm_work(1, T, H), device="cuda") for _ in range(2)]
    outs = (h, y, dx, q, rstd, dw)
    with ccr_mod.Context(0) as c:
        def both(mine, stream=None):
            ccr_mod.ccr_rms_norm(c, [x], [w], y=[y], q=[q], residual=[res], h=[h], rstd=[rstd], stream=stream)
            ccr_mod.ccr_rms_norm_bwd(c, [dy], [h], [w], [rstd], [dx], [dw], work[mine], dh=[dh], stream=stream)

        for t in (x, res, dy, dh):
            t.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both(0)
        side = torch.cuda.Stream()
        for step in range(3):
            for t in (x, res, dy, dh):
                t.copy_(torch.randn(T, H, device="cuda"))
            torch.cuda.synchronize()
            both(1, side)
            side.synchronize()
            want = [t.clone() for t in outs]
            for t in outs:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {step}"


def test_two_calls_at_once(ccr_mod):
    """Calls on two streams, each with a work array of its own."""
    import torch
    T, H = 3000, 1024
    g = gen(9)
    sets = [[rnd(g, T, H).bfloat16() for _ in range(2)] for _ in range(2)]
    w, rstd = torch.ones(H, device="cuda"), torch.ones(T, device="cuda")
    dx = [[torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    dw = [[torch.empty(H, device="cuda") for _ in range(2)] for _ in range(2)]
    work = [torch.empty(ccr_mod.ccr_rms_norm_work(1, T, H), device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    with ccr_mod.Context(0) as c:
        for i, (dy, h) in enumerate(sets):
            ccr_mod.ccr_rms_norm_bwd(c, [dy], [h], [w], [rstd], [dx[0][i]], [dw[0][i]], work[0])
        torch.cuda.synchronize()
        for _ in range(5):
            for i, (dy, h) in enumerate(sets):
                ccr_mod.ccr_rms_norm_bwd(c, [dy], [h], [w], [rstd], [dx[1][i]], [dw[1][i]], work[i],
                                         stream=streams[i])
        torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(dx[0][i], dx[1][i]) and torch.equal(dw[0][i], dw[1][i])


def test_offsets_past_32_bits(ccr_mod):
    """The last rows lie past 2^32 bytes from the first."""
    import torch
    T, H = 300000, 8192
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    say("norm past 32-bit offsets")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, y = torch.zeros(T, H, **bf), torch.empty(T, H, **bf)
    x[-3:] = torch.randn(3, H, device="cuda")
    q = torch.empty(T, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    w = torch.ones(H, **bf)
    rstd, dw, sdw = torch.empty(T, device="cuda"), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    work = torch.empty(ccr_mod.ccr_rms_norm_work(1, T, H), device="cuda")
    sx = x[-3:].clone()
    sy, sdx, srstd = torch.empty_like(sx), torch.empty_like(sx), torch.empty(3, device="cuda")
    sq = torch.empty(3, q.shape[1], dtype=torch.uint8, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_rms_norm(c, [x], [w], y=[y], q=[q], rstd=[rstd])
        ccr_mod.ccr_rms_norm(c, [sx], [w], y=[sy], q=[sq], rstd=[srstd])
        torch.cuda.synchronize()
        assert torch.equal(y[-3:], sy) and torch.equal(q[-3:], sq) and torch.equal(rstd[-3:], srstd)
        assert not bool(y[:-3].any()) and not bool(q[:-3].any())
        ccr_mod.ccr_rms_norm_bwd(c, [x], [x], [w], [rstd], [y], [dw], work)
        ccr_mod.ccr_rms_norm_bwd(c, [sx], [sx], [w], [srstd], [sdx], [sdw], work)
        torch.cuda.synchronize()
    assert torch.equal(y[-3:], sdx) and not bool(y[:-3].any())
    assert bool(((dw - sdw).abs() <= 8 * U * (sx.double() ** 2 * srstd.double()[:, None]).sum(0)).all())


def test_empty_and_refusals(ccr_mod):
    import torch
    T, H = 4, 64
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, res, y, h = (torch.full((T, H), 7.0, **bf) for _ in range(4))
    w = torch.ones(H, **bf)
    q = torch.full((T, r8.row_bytes(H)), 9, dtype=torch.uint8, device="cuda")
    rstd, dw = torch.ones(T, device="cuda"), torch.full((H,), 5.0, device="cuda")
    work = torch.empty(ccr_mod.ccr_rms_norm_work(1, T, H), device="cuda")
    E = ccr_mod.CcrError
    with ccr_mod.Context(0) as c:
        norm = lambda *a, **k: ccr_mod.ccr_rms_norm(c, *a, **k)
        bwd = lambda *a, **k: ccr_mod.ccr_rms_norm_bwd(c, *a, **k)
        norm([x[:0]], [w], y=[y[:0]])
        for args, kw, err, word in [
                (([x], [w]), {}, E, "y and q"),
                (([x], [w]), dict(y=[x]), E, "overlap"),
                (([x], [w]), dict(y=[y], residual=[res]), E, "together"),
                (([x], [w]), dict(y=[y], residual=[res], h=[y]), E, "overlap"),
                (([x], [w]), dict(y=[y], eps=-1.0), E, "eps"),
                (([x], [w]), dict(y=[y], eps=float("nan")), E, "eps"),
                (([x], [w[:-1]]), dict(y=[y]), ValueError, "shape"),
                (([x], [w]), dict(q=[q[:, :-1]]), ValueError, "shape"),
                (([x], [w]), dict(y=[y.float()]), TypeError, "y"),
                (([x.half()], [w]), dict(y=[y]), TypeError, "dtype"),
                (([x.t()], [w]), dict(y=[y]), ValueError, "shape|contiguous"),
                (([x[:, :4].contiguous()], [w[:4].contiguous()]), dict(y=[y[:, :4].contiguous()]), E, "16 bytes")]:
            with pytest.raises(err, match=word):
                norm(*args, **kw)
        with pytest.raises(E, match="overlap"):
            bwd([x], [res], [w], [rstd], [x], [dw], work)
        with pytest.raises(E, match="overlap"):
            bwd([x], [res], [w], [rstd], [y], [work[:H]], work)
        with pytest.raises(ValueError, match="shape"):
            bwd([x], [res], [w], [rstd], [y], [dw], work[:-1])
        torch.cuda.synchronize()
        assert all(bool((t == 7.0).all()) for t in (x, res, y, h)) and bool((q == 9).all()) and bool((dw == 5).all())
        # no row: the weight's gradient is 0, or stays
        bwd([x[:0]], [x[:0]], [w], [rstd[:0]], [y[:0]], [dw], None, accumulate=True)
        torch.cuda.synchronize()
        assert bool((dw == 5).all())
        bwd([x[:0]], [x[:0]], [w], [rstd[:0]], [y[:0]], [dw], None)
        torch.cuda.synchronize()
    assert not bool(dw.any())
