"""8-bit rows on the GPU: bytes equal to the format's definition, and the experts'
products on them against 64-bit references."""
import numpy as np
import pytest

import rows8_helpers as r8
from gpu_helpers import say, torch_cuda
from operator_helpers import Guarded, HALF, counts_of, inside_nan, tdtype

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


def round_trip(ccr, xs, dt, seed=0):
    """Quantised bytes equal to the definition's, and what comes back exact."""
    import torch
    H = xs[0].shape[-1]
    say(f"rows8 {[tuple(x.shape) for x in xs]} {dt}")
    xs = [inside_nan(x.to(tdtype(dt)).cuda()) for x in xs]
    q = [Guarded((*x.shape[:-1], r8.row_bytes(H)), torch.uint8, fill=9) for x in xs]
    y = [Guarded(x.shape, torch.bfloat16) for x in xs]
    z = [Guarded(x.shape, torch.float32) for x in xs]
    assert ccr.ccr_q8_row_bytes(H) == r8.row_bytes(H)
    with ccr.Context(0) as c:
        ccr.ccr_quantize_rows(c, xs, [o.t for o in q])
        ccr.ccr_dequantize_rows(c, [o.t for o in q], [o.t for o in y])
        ccr.ccr_dequantize_rows(c, [o.t for o in q], [o.t for o in z])
        torch.cuda.synchronize()
    for x, a, b, d in zip(xs, q, y, z):
        assert a.intact() and b.intact() and d.intact()
        rows = a.t.cpu().numpy()
        assert np.array_equal(rows, r8.pack(x.double().cpu().numpy()))
        want = torch.from_numpy(r8.unpack(rows, H)[0])
        assert torch.equal(d.t.cpu().nan_to_num(7.0), want.float().nan_to_num(7.0))
        assert torch.equal(b.t.cpu().nan_to_num(7.0), want.bfloat16().nan_to_num(7.0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shapes", [[(1, 8)], [(1, 2048)], [(3, 24), (0, 24), (5, 24)], [(2, 3, 520)], [(7, 1032)],
                                    [(1, 4104)], [(300, 128)], [(65, 256), (1, 256)], [(2, 16392)], [(33, 40)] * 64])
def test_round_trip(ccr_mod, shapes, dt):
    import torch
    g = torch.Generator()
    g.manual_seed(len(shapes) + shapes[0][-1])
    round_trip(ccr_mod, [torch.randn(s, generator=g) * 3 for s in shapes], dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_blocks_at_every_border(ccr_mod, dt):
    """Magnitudes over the whole range of fp32, blocks whose largest value lies at,
    just below and just above 448 times a power of two, ties between two values of
    e4m3, subnormal values, zeros and negative zeros, infinities and NaN."""
    import torch
    g = torch.Generator()
    g.manual_seed(1)
    H = 128
    rows = []
    for e in range(-149, 128, 5):
        rows.append(torch.randn(H, generator=g, dtype=torch.float64) * 2.0 ** min(e, 125))
    for e in (-120, -20, 0, 60):
        top = 448 * 2.0 ** e
        for t in (top, top * (1 - 2.0 ** -24), top * (1 + 2.0 ** -23), top * (1 + 2.0 ** -7)):
            r = torch.randn(H, generator=g, dtype=torch.float64) * top / 500
            r[::32] = t
            rows.append(r.clamp(-t, t))
    grid = torch.from_numpy(r8.VALUES[:127])
    ties = torch.cat([grid, (grid[1:] + grid[:-1]) / 2])
    ties = torch.cat([ties, -ties])
    for i in range(0, len(ties) - 31, 31):
        r = torch.zeros(H, dtype=torch.float64)
        r[:31] = ties[i:i + 31]
        r[31] = 448
        rows.append(r)
    x = torch.stack(rows).float()
    x[0] = 0
    x[1] = -0.0
    x[2, 3], x[3, 40], x[4, 127] = float("inf"), float("nan"), float("-inf")
    round_trip(ccr_mod, [x], dt)


def experts_ref(exp, w, rows, R, E, H):
    """fp64 results, and for every result what the matrix instruction may lose: the
    products of 16 neighbours keep 13 bits below the largest of them (each of the
    16 is off by less than 2^-13 of it), and the fp32 sums half a unit an addition."""
    import torch
    eloc = E // R
    res, lost = [], []
    for d in range(R):
        at, parts, offs = 0, [], []
        x, ww = (torch.from_numpy(r8.unpack(t.cpu().numpy(), H)[0]) for t in (exp[d], w[d]))
        pad = (0, -H % 128)
        for l in range(eloc):
            n = int(rows[d * eloc + l])
            a = torch.nn.functional.pad(x[at:at + n], pad).unflatten(-1, (-1, 16))
            b = torch.nn.functional.pad(ww[l], pad).unflatten(-1, (-1, 16))
            parts.append(x[at:at + n] @ ww[l].t())
            off = torch.zeros_like(parts[-1])
            mag = x[at:at + n].abs() @ ww[l].abs().t()
            for k in range(a.shape[1]):
                off += 16 * 2.0 ** -13 * (a[:, None, k].abs() * b[None, :, k].abs()).amax(-1)
            offs.append(off + (H / 128 + 8) * U * mag)
            at += n
        res.append(torch.cat(parts))
        lost.append(torch.cat(offs))
    return res, lost


def run_experts(ccr, exp, w, counts, H, F, more=0):
    """out[d] between guards, with `more` rows behind the last."""
    import torch
    R = len(w)
    out = [Guarded((len(x) + more, F), torch.bfloat16, fill=7.0) for x in exp]
    with ccr.Context(0) as c:
        ccr.ccr_moe_experts_q8(c, exp, w, counts, H, [o.t for o in out])
        torch.cuda.synchronize()
    for x, o in zip(exp, out):
        assert o.intact() and bool((o.t[len(x):] == 7.0).all())
    return [o.t[:len(x)] for x, o in zip(exp, out)]


def packed(x):
    import torch
    return torch.from_numpy(r8.pack(x)).cuda()


CASES = [  # R, rows per expert, H, F
    (1, [1], 8, 8), (1, [1, 1, 1], 2048, 72), (1, [0, 3], 24, 40), (2, [5, 0, 17, 64], 264, 136),
    (1, [130, 1], 512, 264), (4, [9, 33, 2, 0, 65, 7, 128, 40], 136, 520), (1, [300, 70], 640, 392),
    (1, [16] * 8, 1032, 8), (2, [0, 0, 1, 0], 4104, 16), (1, [700], 128, 1032), (1, [1030, 300], 1032, 520)]


@pytest.mark.parametrize("R,rows,H,F", CASES)
def test_whole_numbers_are_exact(ccr_mod, R, rows, H, F):
    """Small whole numbers times powers of two that differ from block to block:
    every product and sum is exact, so the results are equal bit for bit, whatever
    the lane, block or step a value goes through."""
    import torch
    rng = np.random.default_rng(H * F)
    E = len(rows)
    counts = counts_of(rows, R, E, rng)
    say(f"experts8 exact R={R} rows={rows} H={H} F={F}")

    def values(n):
        # sparse, so that sums stay below 2^8 and bf16 holds them; the two sides'
        # scales of a block of 32 cancel
        v = rng.integers(-3, 4, size=(n, H)) * (rng.random((n, H)) < min(1.0, 12 / H))
        return v.astype(np.float64)

    scale = np.repeat(rng.integers(-6, 7, size=-(-H // 32)), 32)[:H]
    eloc = E // R
    per = [sum(rows[d * eloc:(d + 1) * eloc]) for d in range(R)]
    xs = [values(n) for n in per]
    ws = [np.stack([values(F) for _ in range(eloc)]) for _ in range(R)]
    exp = [packed(np.ldexp(x, scale)) for x in xs]
    w = [packed(np.ldexp(x, -scale)) for x in ws]
    got = run_experts(ccr_mod, exp, w, counts, H, F, more=3)
    for d in range(R):
        at = 0
        for l in range(eloc):
            n = rows[d * eloc + l]
            want = xs[d][at:at + n] @ ws[d][l].T
            assert np.abs(want).max(initial=0) <= 256
            assert np.array_equal(got[d][at:at + n].float().cpu().numpy(), want)
            at += n


@pytest.mark.parametrize("H", [72, 200, 344, 520, 1160])
def test_many_rows_are_exact(ccr_mod, H):
    """The same over several rounds of the largest tiles, of 1 to 10 steps, with rows
    and columns that end inside a tile: rows of -1, 0 and 1 against at most 60 values
    of up to 4, in blocks of different powers of two."""
    import torch
    rng = np.random.default_rng(H)
    rows, F = [12000, 0, 9001, 130, 257, 5000], 2040
    counts = counts_of(rows, 1, len(rows), rng)
    say(f"experts8 rows={rows} H={H} F={F}")
    scale = np.repeat(rng.integers(-3, 4, size=-(-H // 32)), 32)[:H]
    x = rng.integers(-1, 2, size=(sum(rows), H)).astype(np.float32)
    w = np.zeros((len(rows), F, H), np.float32)
    at = rng.integers(0, H, size=(len(rows), F, 60))
    np.put_along_axis(w, at, rng.integers(-4, 5, size=at.shape).astype(np.float32), 2)
    got, = run_experts(ccr_mod, [packed(np.ldexp(x, scale))], [packed(np.ldexp(w, -scale))], counts, H, F, more=3)
    first = 0
    for e, n in enumerate(rows):
        want = torch.from_numpy(x[first:first + n]).cuda() @ torch.from_numpy(w[e]).cuda().t()  # whole numbers
        assert torch.equal(got[first:first + n].float(), want)
        first += n


@pytest.mark.parametrize("R,rows,H,F", CASES)
def test_against_the_reference(ccr_mod, R, rows, H, F):
    import torch
    rng = np.random.default_rng(H + F)
    E = len(rows)
    counts = counts_of(rows, R, E, rng)
    say(f"experts8 R={R} rows={rows} H={H} F={F}")
    eloc = E // R
    per = [sum(rows[d * eloc:(d + 1) * eloc]) for d in range(R)]
    exp = [packed(rng.normal(size=(n, H)) * np.exp(rng.normal(size=(1, H)))) for n in per]
    w = [packed(rng.normal(size=(eloc, F, H)) / H ** 0.5) for _ in range(R)]
    got = run_experts(ccr_mod, exp, w, counts, H, F)
    want, lost = experts_ref(exp, w, rows, R, E, H)
    for g, x, m in zip(got, want, lost):
        g = g.double().cpu()
        assert bool(((g - x).abs() <= HALF["bf16"] * x.abs() * (1 + HALF["bf16"]) + 1.01 * m).all())


@pytest.mark.parametrize("rows,H,F", [([900, 0, 3000, 513], 1024, 1000), ([2000], 4096, 2048), ([40] * 16, 2048, 512),
                                      ([5000, 3], 384, 776)])
def test_error_of_normal_rows(ccr_mod, rows, H, F):
    """Every product is off by at most 2^-13 of the largest of 16, in no preferred
    direction: over H normal products, whose largest of 16 is about 4.5, by 2^-13
    4.5 sqrt(H) against results of sqrt(H), together with the bf16 rounding (2^-9 /
    sqrt 3 relative, taken over the values' mantissas) below 2^-9."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    E = len(rows)
    say(f"experts8 normal rows={rows} H={H} F={F}")
    n = sum(rows)
    exp = torch.empty(n, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    w = torch.empty(E, F, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    x, ww = torch.randn(n, H, generator=g, device="cuda"), torch.randn(E, F, H, generator=g, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_quantize_rows(c, [x], [exp])
        ccr_mod.ccr_quantize_rows(c, [ww], [w])
        ccr_mod.ccr_dequantize_rows(c, [exp], [x])
        ccr_mod.ccr_dequantize_rows(c, [w], [ww])
        torch.cuda.synchronize()
    got = run_experts(ccr_mod, [exp], [w], np.array([rows], np.int64), H, F)[0]
    at = 0
    for e, k in enumerate(rows):
        if k == 0:
            continue
        want = x[at:at + k].double() @ ww[e].double().t().contiguous()
        err = got[at:at + k].double() - want
        assert float(err.square().mean().sqrt()) <= 2.0 ** -9 * float(want.square().mean().sqrt())
        # and nowhere far off: fourteen times that anywhere would be a lost block
        assert float(err.abs().max()) <= 2.0 ** -5 * float(want.abs().max())
        at += k


def test_not_finite_blocks(ccr_mod):
    """A block that stands for NaN makes its row's results NaN, in the rows its
    column's; zeros against anything finite stay 0."""
    import torch
    H, F = 256, 40
    rng = np.random.default_rng(3)
    x, w = rng.normal(size=(5, H)), rng.normal(size=(1, F, H))
    x[1, 70] = np.inf
    x[2] = 0
    w[0, 7, 200] = np.nan
    got = run_experts(ccr_mod, [packed(x)], [packed(w)], np.array([[5]], np.int64), H, F)[0]
    bad = torch.zeros(5, F, dtype=torch.bool, device="cuda")
    bad[1] = True
    bad[:, 7] = True
    assert torch.equal(got.isnan(), bad)
    assert not bool(got[2][~bad[2]].any())


def test_scales_at_the_ends_of_their_range(ccr_mod):
    """Scales of 2^-127 against 2^113: their product is what counts."""
    import torch
    H, F = 128, 16
    rng = np.random.default_rng(4)
    x, w = rng.integers(-3, 4, size=(4, H)).astype(float), rng.integers(-3, 4, size=(1, F, H)).astype(float)
    x[:, ::32], w[:, :, ::32] = 3, 3
    got = run_experts(ccr_mod, [packed(np.ldexp(x, -120))], [packed(np.ldexp(w, 120))], np.array([[4]], np.int64), H, F)
    want = torch.from_numpy(x @ w[0].T)
    assert torch.equal(got[0].cpu(), want.bfloat16())


def test_streams_and_graph_replays(ccr_mod):
    import torch
    H, F, rows = 384, 136, [20, 0, 33, 7]
    n = sum(rows)
    counts = np.array([rows], np.int64)
    x, w = torch.empty(n, H, device="cuda"), torch.empty(4, F, H, device="cuda")
    x8 = torch.empty(n, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    w8 = torch.empty(4, F, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    back, out = torch.empty_like(x), torch.empty(n, F, dtype=torch.bfloat16, device="cuda")
    with ccr_mod.Context(0) as c:
        def all_(stream=None):
            ccr_mod.ccr_quantize_rows(c, [x], [x8], stream=stream)
            ccr_mod.ccr_quantize_rows(c, [w], [w8], stream=stream)
            ccr_mod.ccr_dequantize_rows(c, [x8], [back], stream=stream)
            ccr_mod.ccr_moe_experts_q8(c, [x8], [w8], counts, H, [out], stream=stream)

        x.zero_()
        w.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            all_()
        side = torch.cuda.Stream()
        for step in range(3):
            x.copy_(torch.randn(n, H, device="cuda"))
            w.copy_(torch.randn(4, F, H, device="cuda"))
            torch.cuda.synchronize()
            all_(side)
            side.synchronize()
            want = [t.clone() for t in (x8, w8, back, out)]
            for t in (x8, w8, back, out):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((x8, w8, back, out), want)), f"replay {step}"


def test_offsets_past_32_bits(ccr_mod):
    """Rows whose last lies past 2^32 bytes from the first."""
    import torch
    n, H, F = 540000, 8192, 16
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    say("rows8 past 32-bit offsets")
    x = torch.zeros(n, H, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, H, device="cuda")
    q = torch.empty(n, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    w = torch.empty(2, F, q.shape[1], dtype=torch.uint8, device="cuda")
    out, small = torch.empty(n, F, dtype=torch.bfloat16, device="cuda"), torch.empty(3, F, dtype=torch.bfloat16, device="cuda")
    ww = torch.randn(2, F, H, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_quantize_rows(c, [x], [q])
        ccr_mod.ccr_quantize_rows(c, [ww], [w])
        ccr_mod.ccr_moe_experts_q8(c, [q], [w], np.array([[5, n - 5]], np.int64), H, [out])
        ccr_mod.ccr_moe_experts_q8(c, [q[-3:]], [w], np.array([[0, 3]], np.int64), H, [small])
        want = x[-3:].clone()
        ccr_mod.ccr_dequantize_rows(c, [q], [x])
        torch.cuda.synchronize()
    assert np.array_equal(q[-3:].cpu().numpy(), r8.pack(want.double().cpu().numpy()))
    assert not bool(x[:-3].any()) and not bool(out[:-3].any())
    # the same products, perhaps of another tile
    assert bool(((out[-3:].double() - small.double()).abs() <= 2 * HALF["bf16"] * small.double().abs() + 1e-3).all())


def test_empty_and_refusals(ccr_mod):
    import torch
    H, F = 64, 16
    x = torch.ones(3, H, dtype=torch.bfloat16, device="cuda")
    q = torch.full((3, r8.row_bytes(H)), 9, dtype=torch.uint8, device="cuda")
    w = torch.zeros(2, F, r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    out = torch.full((3, F), 7.0, dtype=torch.bfloat16, device="cuda")
    E = ccr_mod.CcrError
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_quantize_rows(c, [x[:0]], [q[:0]])
        ccr_mod.ccr_dequantize_rows(c, [q[:0]], [x[:0]])
        ccr_mod.ccr_moe_experts_q8(c, [q[:0]], [w], [[0, 0]], H, [out[:0]])
        for call, err, word in [
                (lambda: ccr_mod.ccr_quantize_rows(c, [x], [q[:, :-1]]), ValueError, "shape"),
                (lambda: ccr_mod.ccr_quantize_rows(c, [x], [q[:2]]), ValueError, "shape"),
                (lambda: ccr_mod.ccr_quantize_rows(c, [x], [q.char()]), TypeError, "q"),
                (lambda: ccr_mod.ccr_quantize_rows(c, [x.half()], [q]), TypeError, "dtype"),
                (lambda: ccr_mod.ccr_quantize_rows(c, [x, x], [q, q]), E, "overlap"),
                (lambda: ccr_mod.ccr_dequantize_rows(c, [q, q], [x, x]), E, "overlap"),
                (lambda: ccr_mod.ccr_quantize_rows(c, [x[:, :4].contiguous()], [q]), E, "16 bytes"),
                (lambda: ccr_mod.ccr_moe_experts_q8(c, [q], [w], [[1, 2]], H + 128, [out]), ValueError, "shape"),
                (lambda: ccr_mod.ccr_moe_experts_q8(c, [q], [w], [[1, 3]], H, [out]), ValueError, "shape"),
                (lambda: ccr_mod.ccr_moe_experts_q8(c, [q], [w], [[-1, 3]], H, [out]), E, "< 0"),
                (lambda: ccr_mod.ccr_moe_experts_q8(c, [q], [w], [[1, 2]], H, [out.float()]), TypeError, "out"),
                (lambda: ccr_mod.ccr_moe_experts_q8(c, [q], [w[:, :3].contiguous()], [[1, 2]], H,
                                                    [out[:, :3].contiguous()]), E, "16 bytes"),
                (lambda: ccr_mod.ccr_moe_experts_q8(c, [q], [w], [[1, 2]], H, [q.view(-1)[:96].view(torch.bfloat16)
                                                                              .view(3, F)]), E, "overlap")]:
            with pytest.raises(err, match=word):
                call()
        torch.cuda.synchronize()
    assert bool((q == 9).all()) and bool((out == 7.0).all()) and bool((x == 1).all())
