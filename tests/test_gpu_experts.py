"""GPU parity of the experts' products with a 64-bit reference.

Whole-number inputs small enough that every sum is exact in fp32 have one
right answer, whatever the order of the sums: those cases compare bit for bit.
Random inputs compare within the error of the sums, derived at the test."""
import numpy as np
import pytest

from gpu_helpers import say, torch_cuda
from operator_helpers import Guarded, HALF, counts_of, experts_ref, inside_nan, tdtype

pytestmark = pytest.mark.gpu

OPS = ["product", "dgrad", "wgrad"]


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


def make(op, dt, rows, R, H, F, seed, whole):
    """(ecnt, first operand, second operand, output shapes) per rank."""
    import torch
    E = len(rows)
    eloc = E // R
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def values(*shape):
        if whole:
            v = torch.randint(-3, 4, shape, generator=g, device="cuda").float()
        else:
            v = torch.randn(shape, generator=g, device="cuda")
        return inside_nan(v.to(tdtype(dt)))

    tot = [int(sum(rows[d * eloc:(d + 1) * eloc])) for d in range(R)]
    a = [values(t, H if op == "product" else F) for t in tot]
    if op == "wgrad":
        b = [values(t, H) for t in tot]
        shapes = [(eloc, F, H)] * R
    else:
        b = [values(eloc, F, H) for _ in range(R)]
        shapes = [(t, F if op == "product" else H) for t in tot]
    return counts_of(rows, R, E, rng), a, b, shapes


def call(ccr, c, op, a, b, ecnt, out, **kw):
    if op == "product":
        ccr.ccr_moe_experts(c, a, b, ecnt, out, **kw)
    elif op == "dgrad":
        ccr.ccr_moe_experts_dgrad(c, a, b, ecnt, out, **kw)
    else:
        ccr.ccr_moe_experts_wgrad(c, b, a, ecnt, out, **kw)


def check(ccr, op, dt, rows, R, H, F, seed=0, whole=True, out_dt=None, accumulate=False):
    import torch
    out_dt = out_dt or dt
    say(f"experts {op} {dt}->{out_dt} rows={list(rows)[:12]} R={R} H={H} F={F} whole={whole} acc={accumulate}")
    ecnt, a, b, shapes = make(op, dt, rows, R, H, F, seed, whole)
    fill = 3.0 if accumulate else float("nan")
    outs = [Guarded(s, tdtype(out_dt), fill) for s in shapes]
    with ccr.Context(0) as c:
        call(ccr, c, op, a, b, ecnt, [o.t for o in outs], **({"accumulate": True} if accumulate else {}))
        torch.cuda.synchronize()
    ref, mag = experts_ref(op, a, b, rows, R, len(rows))
    inner = {"product": H, "dgrad": F, "wgrad": max(list(rows) + [1])}[op]
    for d in range(R):
        assert outs[d].intact(), f"rank {d}: a guard byte changed"
        want = ref[d] + (3.0 if accumulate else 0.0)
        got = outs[d].t
        if whole:
            assert torch.equal(got, want.to(tdtype(out_dt))), f"rank {d} differs"
        else:
            # each of the `inner` fp32 additions and the adding of the old value is
            # off by at most one unit (2^-23) of a partial sum, which the sum of the
            # products' magnitudes bounds; then one rounding to the output type
            tol = HALF[out_dt] * want.abs() + (inner + 1) * 2.0 ** -23 * (mag[d] + 3.0 * accumulate) * 1.01
            assert bool(((got.double() - want).abs() <= tol).all()), f"rank {d} out of tolerance"
    return outs


ROWS = {
    "one row": [1],
    "no row at all": [0, 0],
    "one expert of four": [0, 0, 5, 0],
    "single tokens": [1, 0, 1, 1, 0, 0, 1, 2],
    "around sixteen": [15, 16, 17, 0],
    "around thirty-two": [31, 32, 33, 48],
    "around a tile": [63, 64, 65, 127, 128, 129],
    "ragged": [300, 0, 1, 257, 77, 512, 0, 9],
}


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS.values(), ids=ROWS.keys())
@pytest.mark.parametrize("H,F", [(8, 8), (72, 136), (264, 520), (1032, 200)])
def test_whole_numbers_bitwise(ccr_mod, op, dt, rows, H, F):
    check(ccr_mod, op, dt, rows, 1, H, F, seed=H + F + len(rows))


MID = [200, 129, 255, 0, 190, 199, 256, 250, 240]
LONG = [2000, 1999, 1801, 2048, 2001, 1793, 1900, 2047]
MANY = [4096, 4000, 0, 3999, 1, 4095, 257, 4097, 255, 3000]


@pytest.mark.parametrize("op,dt,out_dt,rows,H,F", [
    # tiles of 128 and of 256, the last of a row of tiles and of a contraction partial
    ("product", "bf16", "bf16", MID, 2056, 2040), ("dgrad", "bf16", "bf16", MID, 2040, 2056),
    ("product", "bf16", "bf16", LONG, 1032, 1000), ("dgrad", "bf16", "bf16", LONG, 1000, 1032),
    # more than one round of tiles, a contraction of few steps
    ("product", "bf16", "bf16", MANY, 264, 2056), ("dgrad", "bf16", "bf16", MANY, 2056, 264),
    ("product", "bf16", "bf16", MANY, 8, 2056), ("dgrad", "bf16", "bf16", MANY, 2056, 72),
    ("wgrad", "bf16", "f32", LONG, 1000, 1032), ("wgrad", "bf16", "bf16", LONG + [0, 1], 1032, 1032),
    # unequal weight gradients in several rounds
    ("wgrad", "bf16", "f32", [400, 399, 0, 1, 64, 65, 700, 128] * 2, 2040, 1400),
    ("wgrad", "bf16", "bf16", [400, 399, 0, 1, 64, 65, 700, 128] * 2, 2040, 1400),
    ("product", "f32", "f32", [4095, 4090], 1028, 2044), ("dgrad", "f32", "f32", [4095, 4090], 2044, 1028),
    ("wgrad", "f32", "f32", [2000, 2009, 1000], 2044, 2040),
])
def test_large_tiles_bitwise(ccr_mod, op, dt, out_dt, rows, H, F):
    check(ccr_mod, op, dt, rows, 1, H, F, out_dt=out_dt, seed=H + F)


@pytest.mark.parametrize("out_dt", ["f32", "bf16"])
def test_large_accumulation_bitwise(ccr_mod, out_dt):
    check(ccr_mod, "wgrad", "bf16", [400, 399, 0, 1, 64, 65, 700, 128] * 2, 2, 2040, 1400, out_dt=out_dt,
          accumulate=True)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [[2, 0, 1], [270, 0, 5]], ids=["few rows", "more than a tile"])
@pytest.mark.parametrize("H,F", [(1 << 20, 8), (8, 1 << 20)])
def test_longest_rows_bitwise(ccr_mod, op, dt, rows, H, F):
    # 9 x 2^20 < 2^24: every sum is exact
    check(ccr_mod, op, dt, rows, 1, H, F, seed=5)


@pytest.mark.parametrize("op", OPS)
def test_offsets_past_32_bits(ccr_mod, op):
    """Rows, weights and results that lie past 2^32 bytes from their buffer's
    first byte: expert 1's are compared, expert 0's are many."""
    import torch
    H, F, n0, n1 = 2048, 2048, 1100000, 300
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    say(f"experts {op} past 32-bit offsets")
    x = torch.zeros(n0 + n1, H if op == "product" else F, dtype=torch.bfloat16, device="cuda")
    x[n0:] = torch.randint(-3, 4, (n1, x.shape[1]), device="cuda").to(torch.bfloat16)
    ecnt = np.array([[n0, n1]], np.int64)
    with ccr_mod.Context(0) as c:
        if op == "wgrad":
            y = torch.ones(n0 + n1, H, dtype=torch.bfloat16, device="cuda")
            y[n0:] = torch.randint(-3, 4, (n1, H), device="cuda").to(torch.bfloat16)
            dw = torch.empty(2, F, H, device="cuda")
            ccr_mod.ccr_moe_experts_wgrad(c, [y], [x], ecnt, [dw])
            torch.cuda.synchronize()
            assert torch.equal(dw[1], (x[n0:].double().t() @ y[n0:].double()).float())
            assert not bool(dw[0].any())
            return
        w = torch.randint(-3, 4, (2, F, H), device="cuda").to(torch.bfloat16)
        out = torch.empty(n0 + n1, F if op == "product" else H, dtype=torch.bfloat16, device="cuda")
        call(ccr_mod, c, op, [x], [w], ecnt, [out])
        torch.cuda.synchronize()
        w1 = w[1].double().t() if op == "product" else w[1].double()
        assert torch.equal(out[n0:], (x[n0:].double() @ w1).to(torch.bfloat16))
        assert not bool(out[:n0].any())


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_several_ranks_bitwise(ccr_mod, op, dt):
    check(ccr_mod, op, dt, [5, 0, 130, 64, 0, 0, 33, 200], 4, 136, 264, seed=3)  # rank 2 has no row


@pytest.mark.parametrize("op", OPS)
def test_fp32_rows_of_four_values(ccr_mod, op):
    check(ccr_mod, op, "f32", [3, 70, 0, 129], 2, 4, 12)
    check(ccr_mod, op, "f32", [3, 70, 0, 129], 2, 132, 68)


@pytest.mark.parametrize("op", OPS)
def test_more_experts_than_one_launch_lists(ccr_mod, op):
    rng = np.random.default_rng(9)
    check(ccr_mod, op, "bf16", list(rng.integers(0, 20, 250)), 2, 40, 24)


# one small output of a long sum, which the waves of a workgroup share by steps
# of 32 (fp32) or 64 values: fewer steps than waves, steps that do not go round
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("long", [8, 32, 40, 64, 72, 128, 160, 192, 200, 256, 264, 328, 1288, 8200])
def test_long_sums_of_few_outputs_bitwise(ccr_mod, op, dt, long):
    if op == "wgrad":
        check(ccr_mod, op, dt, [long, 0, long - 3], 1, 40, 24, seed=long)
        check(ccr_mod, op, dt, [long], 1, 24, 40, seed=long, out_dt="f32", accumulate=True)
    else:
        H, F = (long, 40) if op == "product" else (40, long)
        check(ccr_mod, op, dt, [1, 0, 19], 1, H, F, seed=long)


@pytest.mark.parametrize("op,dt,rows,H,F", [
    ("product", "bf16", [700, 1300, 0, 2500], 1024, 768),
    ("dgrad", "bf16", [700, 1300, 0, 2500], 768, 1024),
    ("wgrad", "bf16", [700, 1300, 0, 2500], 512, 1024),
    ("product", "bf16", [2, 9, 0, 1], 2048, 1024),
    ("product", "f32", [300, 900], 512, 260),
    ("dgrad", "f32", [300, 900], 260, 512),
    ("wgrad", "f32", [300, 900], 260, 516),
    ("wgrad", "bf16", [40000, 3], 88, 176),
    ("product", "bf16", LONG, 1032, 1000),
    ("wgrad", "bf16", LONG, 1000, 1032),
])
def test_random_values_within_the_sums_error(ccr_mod, op, dt, rows, H, F):
    check(ccr_mod, op, dt, rows, 1, H, F, whole=False, seed=H)


@pytest.mark.parametrize("dt,out_dt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("whole", [True, False])
def test_wgrad_types_and_accumulation(ccr_mod, dt, out_dt, whole):
    rows = [50, 0, 1, 300]
    check(ccr_mod, "wgrad", dt, rows, 2, 136, 72, whole=whole, out_dt=out_dt)
    check(ccr_mod, "wgrad", dt, rows, 2, 136, 72, whole=whole, out_dt=out_dt, accumulate=True)


def test_gradients_against_differences(ccr_mod):
    """<dout, experts(x)> is linear in x and in w: moving one entry of either
    by a step changes it by step times that entry's gradient, exactly in
    whole numbers."""
    import torch
    rows, R, H, F = [5, 0, 37], 1, 16, 24
    ecnt, x, w, _ = make("product", "f32", rows, R, H, F, 1, True)
    n = sum(rows)
    dout = [torch.randint(-3, 4, (n, F), device="cuda").float()]
    with ccr_mod.Context(0) as c:
        dx, dw, y = torch.empty(n, H, device="cuda"), torch.empty(3, F, H, device="cuda"), torch.empty(n, F, device="cuda")
        ccr_mod.ccr_moe_experts_dgrad(c, dout, w, ecnt, [dx])
        ccr_mod.ccr_moe_experts_wgrad(c, x, dout, ecnt, [dw])

        def loss(xs, ws):
            ccr_mod.ccr_moe_experts(c, [xs], [ws], ecnt, [y])
            return float((y.double() * dout[0].double()).sum())

        base = loss(x[0], w[0])
        for i, h in [(0, 0), (4, 15), (5, 3), (41, 9)]:
            moved = x[0].clone()
            moved[i, h] += 2
            assert loss(moved, w[0]) - base == 2 * float(dx[i, h])
        for e, f, h in [(0, 0, 0), (2, 23, 15), (2, 7, 1), (1, 3, 3)]:
            moved = w[0].clone()
            moved[e, f, h] += 2
            assert loss(x[0], moved) - base == 2 * float(dw[e, f, h])


@pytest.mark.parametrize("op", OPS)
def test_values_of_other_rows_do_not_leak(ccr_mod, op):
    """A NaN or an infinity in one expert's rows stays with that expert."""
    import torch
    rows, H, F = [70, 3, 130], 72, 136
    ecnt, a, b, shapes = make(op, "bf16", rows, 1, H, F, 2, True)
    a[0][70:73] = float("nan")
    a[0][72] = float("inf")
    out = torch.empty(shapes[0], dtype=torch.bfloat16, device="cuda")
    with ccr_mod.Context(0) as c:
        call(ccr_mod, c, op, a, b, ecnt, [out])
        torch.cuda.synchronize()
    ref, _ = experts_ref(op, a, b, rows, 1, 3)
    keep = [0, 2] if op == "wgrad" else list(range(70)) + list(range(73, 203))
    assert torch.equal(out[keep], ref[0][keep].to(torch.bfloat16))


@pytest.mark.parametrize("op", OPS)
def test_rows_behind_the_last_are_left(ccr_mod, op):
    import torch
    rows, H, F = [9, 40], 24, 40
    ecnt, a, b, shapes = make(op, "bf16", rows, 1, H, F, 4, True)
    pad = lambda t: torch.cat([t, torch.full((7,) + tuple(t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda")])
    a = [pad(t) for t in a]
    b = [pad(t) for t in b] if op == "wgrad" else b
    n = shapes[0][0]
    extra = 0 if op == "wgrad" else 7
    out = torch.full((n + extra,) + tuple(shapes[0][1:]), 5.0, dtype=torch.bfloat16, device="cuda")
    with ccr_mod.Context(0) as c:
        call(ccr_mod, c, op, a, b, ecnt, [out])
        torch.cuda.synchronize()
    ref, _ = experts_ref(op, a, b, rows, 1, 2)
    assert torch.equal(out[:n], ref[0].to(torch.bfloat16))
    assert bool((out[n:] == 5.0).all())


@pytest.mark.parametrize("op", OPS)
def test_another_stream_and_graph_replays(ccr_mod, op):
    import torch
    rows, H, F = [33, 0, 200, 1], 136, 72
    ecnt, a, b, shapes = make(op, "bf16", rows, 1, H, F, 5, True)
    out = torch.zeros(shapes[0], dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    with ccr_mod.Context(0) as c:
        side.wait_stream(torch.cuda.current_stream())
        call(ccr_mod, c, op, a, b, ecnt, [out], stream=side)
        side.synchronize()
        want = experts_ref(op, a, b, rows, 1, 4)[0][0].to(torch.bfloat16)
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(ccr_mod, c, op, a, b, ecnt, [out])
        for step in range(3):
            a[0].copy_(torch.randint(-3, 4, a[0].shape, device="cuda").to(a[0].dtype))
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            want = experts_ref(op, a, b, rows, 1, 4)[0][0].to(torch.bfloat16)
            assert torch.equal(out, want), f"replay {step}"


def test_runs_with_a_cu_budget_and_under_capture(ccr_mod):
    import torch
    ecnt, a, b, shapes = make("product", "bf16", [40, 5], 1, 72, 40, 6, True)
    out = torch.zeros(shapes[0], dtype=torch.bfloat16, device="cuda")
    with ccr_mod.Context(0, ccr_mod.Config(cu_budget=16)) as c:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ccr_mod.ccr_moe_experts(c, a, b, ecnt, [out])
        graph.replay()
        torch.cuda.synchronize()
    assert torch.equal(out, experts_ref("product", a, b, [40, 5], 1, 2)[0][0].to(torch.bfloat16))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_subnormal_values(ccr_mod, op, dt):
    """Products of subnormal and ordinary values keep their bits: 2^-130 times
    whole numbers, summed exactly, is a multiple of 2^-130 still."""
    import torch
    rows, H, F = [40, 3], 72, 40
    ecnt, a, b, shapes = make(op, dt, rows, 1, H, F, 11, True)
    a[0].mul_(2.0 ** -65).mul_(2.0 ** -65)
    out = torch.empty(shapes[0], device="cuda", dtype=tdtype(dt))
    with ccr_mod.Context(0) as c:
        call(ccr_mod, c, op, a, b, ecnt, [out])
        torch.cuda.synchronize()
    ref = experts_ref(op, a, b, rows, 1, 2)[0][0]
    assert bool((ref != 0).any()) and torch.equal(out, ref.to(tdtype(dt)))


def test_two_streams_at_once(ccr_mod):
    """One context, two streams, calls in flight together: each its own result."""
    import torch
    sets = [make(op, "bf16", rows, 1, 264, 392, 12 + i, True)
            for i, (op, rows) in enumerate([("product", [300, 0, 77]), ("dgrad", [1, 512, 65])])]
    ops = ["product", "dgrad"]
    outs = [torch.zeros(s[3][0], dtype=torch.bfloat16, device="cuda") for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    with ccr_mod.Context(0) as c:
        for _ in range(20):
            for op, (ecnt, a, b, _), o, st in zip(ops, sets, outs, streams):
                call(ccr_mod, c, op, a, b, ecnt, [o], stream=st)
        torch.cuda.synchronize()
    for op, (ecnt, a, b, _), o, rows in zip(ops, sets, outs, ([300, 0, 77], [1, 512, 65])):
        assert torch.equal(o, experts_ref(op, a, b, rows, 1, 3)[0][0].to(torch.bfloat16))


def test_same_bits_every_run(ccr_mod):
    import torch
    for op in OPS:
        ecnt, a, b, shapes = make(op, "bf16", [500, 3, 0, 129], 1, 264, 200, 7, False)
        got = []
        with ccr_mod.Context(0) as c:
            for _ in range(3):
                out = torch.empty(shapes[0], dtype=torch.bfloat16, device="cuda")
                call(ccr_mod, c, op, a, b, ecnt, [out])
                got.append(out)
            torch.cuda.synchronize()
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_refusals(ccr_mod):
    import ctypes

    import torch
    bad = ccr_mod.CCR_ERR_INVALID_ARG
    x = torch.ones(8, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(2, 24, 16, dtype=torch.bfloat16, device="cuda")
    y = torch.full((8, 24), 7.0, dtype=torch.bfloat16, device="cuda")
    ecnt = np.array([[5, 3]], np.int64)
    lib = ccr_mod._lib
    with ccr_mod.Context(0) as c:
        def raw(px=x.data_ptr(), pw=w.data_ptr(), py=y.data_ptr(), counts=ecnt, R=1, E=2, H=16, F=24, dt=1):
            one = lambda p: (ctypes.c_void_p * 1)(p)
            return lib.ccr_moe_experts(c.handle, one(px), one(pw), counts.ctypes.data, R, E, H, F, dt,
                                       one(py), None)

        for kw, word in [(dict(px=0), "NULL"), (dict(px=x.data_ptr() + 2), "aligned"),
                         (dict(counts=np.array([[5, -1]], np.int64)), "< 0"),
                         (dict(counts=np.array([[5, 1 << 30]], np.int64)), "past the end"),
                         (dict(H=12), "16 bytes"), (dict(F=1 << 21), "F ="), (dict(H=0), "H ="),
                         (dict(dt=2), "dtype"), (dict(R=0), "R"), (dict(R=2, E=3), "R"),
                         (dict(py=x.data_ptr()), "overlap")]:
            assert raw(**kw) == bad and word in ccr_mod.ccr_last_error(), (kw, ccr_mod.ccr_last_error())
        assert raw(counts=np.array([[1 << 31, 0]], np.int64)) == ccr_mod.CCR_ERR_UNSUPPORTED
        torch.cuda.synchronize()
        assert bool((y == 7.0).all())
        with pytest.raises(TypeError):
            ccr_mod.ccr_moe_experts(c, [x.float()], [w], ecnt, [y])
        with pytest.raises(ValueError):
            ccr_mod.ccr_moe_experts(c, [x[:7]], [w], ecnt, [y])
        with pytest.raises(ValueError):
            ccr_mod.ccr_moe_experts(c, [x], [w.transpose(1, 2)], ecnt, [y])
        with pytest.raises(ValueError):
            ccr_mod.ccr_moe_experts(c, [x], [w], ecnt[0], [y])
        with pytest.raises(ccr_mod.CcrError):  # bf16 gradients of fp32 rows
            ccr_mod.ccr_moe_experts_wgrad(c, [x.float()], [y.float()], ecnt, [w.clone()])


@pytest.mark.parametrize("op", ["product", "dgrad"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_rows_than_one_launch_covers(ccr_mod, op, dt):
    """2^29 narrow rows of one expert, past the 2^23 - 1 tiles of one launch for
    any tile of up to 64 rows: every result, bit for bit."""
    import torch
    n, w = (1 << 29) + 77, 16 // (4 if dt == "f32" else 2)
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    say(f"experts {op} {dt} {n} rows of {w}")
    x = torch.empty(n, w, dtype=tdtype(dt), device="cuda").random_(0, 4)
    weight = torch.empty(1, w, w, dtype=tdtype(dt), device="cuda").random_(0, 4)
    out = torch.full((n, w), 7.0, dtype=tdtype(dt), device="cuda")  # 9 w at most, exact
    with ccr_mod.Context(0) as c:
        call(ccr_mod, c, op, [x], [weight], [[n]], [out])
        torch.cuda.synchronize()
    m = weight[0].t() if op == "product" else weight[0]
    step = 1 << 26
    for at in range(0, n, step):
        part = x[at:at + step]
        want = torch.zeros_like(part)
        for k in range(w):
            want += part[:, k:k + 1] * m[k]
        assert torch.equal(out[at:at + step], want), f"rows from {at}"


def test_more_weights_than_one_launch_covers(ccr_mod):
    """An fp32 weight gradient of 2^18 x 131,136 from one row: more tiles of 64 x 64
    than one launch covers."""
    import torch
    F, H = 1 << 18, 131136
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GiB")
    say(f"experts wgrad f32 {F} x {H}")
    x = torch.empty(1, H, device="cuda").random_(1, 4)
    dout = torch.empty(1, F, device="cuda").random_(1, 4)
    dw = torch.empty(1, F, H, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_moe_experts_wgrad(c, [x], [dout], [[1]], [dw])
        torch.cuda.synchronize()
    for at in range(0, F, 1 << 14):
        assert torch.equal(dw[0, at:at + (1 << 14)], dout[0, at:at + (1 << 14), None] * x), f"rows from {at}"


@pytest.mark.parametrize("op,dt,rows,H,F,chain", [
    ("product", "f32", 1, 65536, 64, 256), ("product", "f32", 300, 65536, 64, 256),
    ("product", "f32", 700, 65536, 512, 256), ("dgrad", "f32", 1, 64, 65536, 256),
    ("dgrad", "f32", 300, 64, 65536, 256), ("dgrad", "f32", 700, 512, 65536, 256),
    ("wgrad", "f32", 65536, 64, 64, 256), ("wgrad", "f32", 65536, 520, 512, 256),
    ("wgrad", "f32", 65536, 2048, 1024, 256), ("wgrad", "bf16", 131072, 64, 64, 2048),
    ("wgrad", "bf16", 262144, 1032, 1024, 2048), ("wgrad", "bf16", 262144, 4096, 4096, 8192),
    ("wgrad", "bf16", 262144 + 8191, 4104, 4096, 8192)])
def test_error_of_long_sums(ccr_mod, op, dt, rows, H, F, chain):
    """Positive values, whose partial sums grow evenly: an addition at k of n is
    off by at most k / n of half a unit of the result, evenly spread, so the
    RMS error of n additions is below sqrt(n) / 3 half units.  A chain of
    `chain` products has at most as many additions; m chains of equal size, joined one
    after the other, come to sqrt(chain / m) / 3 + sqrt(m) / 3.  The sum in one chain of
    matrix instructions is 4 to 8 times as far off."""
    import torch
    say(f"error of long sums {op} {dt} rows={rows} H={H} F={F}")
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    rnd = lambda *s: (torch.rand(s, generator=g, device="cuda") + 0.5).to(tdtype(dt))
    n = {"product": H, "dgrad": F, "wgrad": rows}[op]
    a = rnd(rows, H if op == "product" else F)
    b = rnd(rows, H) if op == "wgrad" else rnd(1, F, H)
    shape = {"product": (rows, F), "dgrad": (rows, H), "wgrad": (1, F, H)}[op]
    out = torch.empty(shape, dtype=torch.float32, device="cuda")
    with ccr_mod.Context(0) as c:
        call(ccr_mod, c, op, [a], [b], [[rows]], [out])
        torch.cuda.synchronize()
    if op == "wgrad":  # some rows of the weight, over the tile
        some = torch.arange(0, F, max(1, F // 64), device="cuda")
        want, got = a[:, some].double().t() @ b.double(), out[0][some]
    else:
        want = a.double() @ (b[0].double().t() if op == "product" else b[0].double())
        got = out
    m = n / chain
    rms = float(((got.double() - want) / want).pow(2).mean().sqrt())
    bound = 2.0 ** -24 * ((chain / m) ** 0.5 + m ** 0.5) / 3
    say(f"  RMS {rms:.3g}, bound {bound:.3g}")
    assert rms <= bound


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradients_of_several_chains_bitwise(ccr_mod, accumulate):
    # 256 x 256 tiles, inside and at the edge, of one to four chains of 8192 rows
    check(ccr_mod, "wgrad", "bf16", [8191, 8192, 8193, 20000, 0, 16384, 16385, 30000], 2, 2056, 2040, out_dt="f32",
          accumulate=accumulate)


@pytest.mark.parametrize("side", ["first", "second"])
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H,F", [([1], 2048, 1024), ([3, 0, 1, 2], 1028, 520), ([16] * 8, 512, 512),
                                      ([33, 130, 0, 64], 264, 200), ([500] * 4, 1024, 1024),
                                      ([900, 1, 1200], 2048, 1032), ([4095, 4090], 1032, 2048)])
def test_every_bit_of_the_operands_counts(ccr_mod, op, dt, rows, H, F, side):
    """One operand selects: one power of two in the sum of each result, the rest
    zeros.  Every result is then a value of the other operand, all of its bits."""
    import torch
    if dt == "bf16":
        H, F = (H + 7) // 8 * 8, (F + 7) // 8 * 8
    say(f"bits {op} {dt} rows={rows} H={H} F={F} the {side} operand selects")
    g = torch.Generator(device="cuda")
    g.manual_seed(H + F)
    E = len(rows)
    a, b, want = [], [], []
    for n in rows:
        shape_a, shape_b = (n, H if op == "product" else F), (n, H) if op == "wgrad" else (F, H)
        x, y = (torch.randn(s, generator=g, device="cuda").to(tdtype(dt)) for s in (shape_a, shape_b))
        # x as [outputs, summed], y as [summed, outputs]
        X, Y = (x.t() if op == "wgrad" else x), (y.t() if op == "product" else y)
        M, C, N = X.shape[0], X.shape[1], Y.shape[1]
        if C == 0:
            want.append(torch.zeros(M, N, dtype=tdtype(dt), device="cuda"))
        else:
            k = M if side == "first" else N
            pick = torch.randint(0, C, (k,), generator=g, device="cuda")
            power = 2.0 ** torch.randint(-2, 3, (k,), generator=g, device="cuda").to(tdtype(dt))
            at = torch.arange(k, device="cuda")
            if side == "first":
                X.zero_()
                X[at, pick] = power
                want.append(power[:, None] * Y[pick])
            else:
                Y.zero_()
                Y[pick, at] = power
                want.append(X[:, pick] * power)
        a.append(x)
        b.append(y)
    a = torch.cat(a).contiguous()
    if op == "wgrad":
        b, want = torch.cat(b).contiguous(), torch.stack(want).contiguous()
    else:
        b, want = torch.stack(b).contiguous(), torch.cat(want).contiguous()
    out = Guarded(want.shape, tdtype(dt))
    with ccr_mod.Context(0) as c:
        call(ccr_mod, c, op, [inside_nan(a)], [inside_nan(b)], [rows], [out.t])
        torch.cuda.synchronize()
    assert out.intact() and torch.equal(out.t, want)
