"""GPU parity of the gradient norm and of clipping with a 64-bit reference."""
import math

import pytest

from gpu_helpers import say, torch_cuda
from operator_helpers import Guarded, HALF, inside_nan, tdtype

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


def scratch(ccr):
    import torch
    return (torch.full((ccr.CCR_GRAD_WORK,), float("nan"), dtype=torch.float64, device="cuda"),
            torch.full((1,), float("nan"), device="cuda"))


def grads_of(sizes, seed=0, scale=1.0):
    """Tensors of (count, dtype, element offset from a 16-byte boundary)."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [inside_nan((scale * torch.randn(n, generator=g, device="cuda")).to(tdtype(dt)), off)
            for n, dt, off in sizes]


def norm64(grads):
    return math.sqrt(math.fsum(float((x.double() ** 2).sum()) for x in grads))


def close_norm(got, want):
    # the fp64 sum of n squares is off by n 2^-53 at most, far below the rounding
    # of the norm to fp32
    return abs(got - want) <= U * want * 1.01


def check_clip(ccr, grads, max_norm, work, norm, out=None, guards=None):
    import torch
    want = norm64(grads)
    before = [x.clone() for x in grads]
    with ccr.Context(0) as c:
        ccr.ccr_grad_clip(c, grads, max_norm, work, norm, out=out)
        torch.cuda.synchronize()
    assert close_norm(float(norm), want)
    q = min(1.0, max_norm / (want + 1e-6))
    for i, (b, o) in enumerate(zip(before, out if out is not None else grads)):
        dt = "f32" if b.dtype == torch.float32 else "bf16"
        # the norm's rounding, the sum's with 1e-6, the quotient's, the product's
        tol = (4 * U + (HALF[dt] if dt == "bf16" else 0)) * 1.01 * (b.double() * q).abs()
        assert bool(((o.double() - b.double() * q).abs() <= tol).all()), f"tensor {i}"
        if out is not None:
            assert torch.equal(grads[i], b), f"tensor {i}: the input changed"


SIZES = {
    "one value": [(1, "f32", 0)],
    "one bf16 value off a boundary": [(1, "bf16", 3)],
    "short, every offset": [(n, dt, o) for n in (1, 2, 3, 5, 9, 15) for dt, k in (("bf16", 8), ("f32", 4))
                            for o in range(k)],
    "around a tile": [(n * 8 + d, "bf16", o) for n in (2048, 4096) for d in (-1, 0, 1, 9) for o in (0, 5)],
    "mixed": [(100003, "f32", 1), (1, "bf16", 1), (0, "f32", 0), (65536, "bf16", 0), (77777, "bf16", 7)],
    "more than one launch lists": [(37 + i * 5, "bf16" if i % 3 else "f32", i % 4) for i in range(250)],
    "many tiles": [(40_000_001, "bf16", 1), (9_000_000, "f32", 0)],
}


# counts around what one launch lists (200, or 133 with results elsewhere)
for _n in (133, 134, 200, 201, 266, 267, 401):
    SIZES[f"{_n} tensors"] = [(5 + i % 40, "bf16" if i % 3 else "f32", i % 4) for i in range(_n)]
# few tiles of 16 KiB, which one workgroup takes, and the first counts it does not
for _tiles in (2, 5, 9, 10, 11, 12, 13):
    SIZES[f"{_tiles} tiles of one tensor"] = [(_tiles * 4096 - 3, "f32", 0)]
    SIZES[f"{_tiles} tensors"] = [(700 + 3 * i, "bf16" if i % 2 else "f32", i % 4) for i in range(_tiles)]


@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
def test_norm(ccr_mod, sizes):
    import torch
    say(f"grad_norm {sizes[:6]} n={len(sizes)}")
    grads = grads_of(sizes)
    work, norm = scratch(ccr_mod)
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_grad_norm(c, grads, work, norm)
        first = float(norm)
        ccr_mod.ccr_grad_norm(c, grads, work, norm)
        torch.cuda.synchronize()
    assert float(norm) == first
    assert close_norm(first, norm64(grads))


@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
@pytest.mark.parametrize("max_norm", [0.25, 1e6])
@pytest.mark.parametrize("where", ["in place", "apart", "apart at another offset"])
def test_clip(ccr_mod, sizes, max_norm, where):
    import torch
    say(f"grad_clip {sizes[:6]} n={len(sizes)} max={max_norm} {where}")
    grads = grads_of(sizes, seed=1)
    work, norm = scratch(ccr_mod)
    if where == "in place":
        check_clip(ccr_mod, grads, max_norm, work, norm)
        return
    shift = 3 if where == "apart at another offset" else 0
    outs = [Guarded((n,), tdtype(dt), offset_elements=off + shift) for n, dt, off in sizes]
    check_clip(ccr_mod, grads, max_norm, work, norm, out=[o.t for o in outs])
    assert all(o.intact() for o in outs)


def test_work_and_norm_stay_inside(ccr_mod):
    import torch
    grads = grads_of([(3_000_000, "bf16", 1)])
    w, n = Guarded((ccr_mod.CCR_GRAD_WORK,), torch.float64), Guarded((1,), torch.float32)
    check_clip(ccr_mod, grads, 0.5, w.t, n.t)
    assert w.intact() and n.intact()


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_squares_beyond_fp32(ccr_mod, scale):
    """Squares that fp32 cannot hold still give the norm."""
    import torch
    grads = grads_of([(5000, "f32", 0), (777, "bf16", 1)], scale=scale)
    work, norm = scratch(ccr_mod)
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_grad_norm(c, grads, work, norm)
        torch.cuda.synchronize()
    assert close_norm(float(norm), norm64(grads)) and 0 < float(norm) < float("inf")


def test_a_tensor_past_32_bits(ccr_mod):
    """2^32 + 99 bf16 values, the last few of them not zero, clipped in place."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    n = 2 ** 32 + 99
    say("grads past 32-bit counts")
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5000, device="cuda").to(torch.bfloat16)
    x[-5000:] = tail
    x[0] = 3.0
    work, norm = scratch(ccr_mod)
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_grad_clip(c, [x[1:]], 0.5, work, norm)
        torch.cuda.synchronize()
    want = norm64([tail])
    assert close_norm(float(norm), want) and float(x[0]) == 3.0
    q = 0.5 / (want + 1e-6)
    err = (x[-5000:].double() - tail.double() * q).abs()
    assert bool((err <= (HALF["bf16"] + 4 * U) * 1.01 * (tail.double() * q).abs()).all())


def test_neighbours_in_memory(ccr_mod):
    """Views that fill a bucket one after the other, in order, out of order,
    with gaps and of two types, give the same as separate tensors."""
    import torch
    work, norm = scratch(ccr_mod)
    flat = inside_nan(torch.randn(100_000, device="cuda").to(torch.bfloat16), 3)
    cuts = [0, 1, 2, 10, 5000, 5003, 5003, 60_001, 99_999, 100_000]
    views = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
    other = torch.randn(77, device="cuda")
    for grads in (views, views[::-1], views[::2], views[:4] + [other] + views[4:]):
        want = norm64(grads)
        outs = [torch.empty_like(g) for g in grads]
        with ccr_mod.Context(0) as c:
            ccr_mod.ccr_grad_norm(c, grads, work, norm)
            assert close_norm(float(norm), want)
            ccr_mod.ccr_grad_clip(c, grads, 0.5, work, norm, out=outs)
            torch.cuda.synchronize()
        q = 0.5 / (want + 1e-6)
        for g, o in zip(grads, outs):
            half = HALF["f32" if g.dtype == torch.float32 else "bf16"]
            assert bool(((o.double() - g.double() * q).abs() <= (half + 4 * U) * 1.01 * (g.double() * q).abs()).all())


def test_nothing_to_measure(ccr_mod):
    import torch
    work, norm = scratch(ccr_mod)
    with ccr_mod.Context(0) as c:
        for grads in ([], grads_of([(0, "f32", 0), (0, "bf16", 0)])):
            norm.fill_(3.0)
            ccr_mod.ccr_grad_norm(c, grads, work, norm)
            assert float(norm) == 0.0
            norm.fill_(3.0)
            ccr_mod.ccr_grad_clip(c, grads, 1.0, work, norm)
            assert float(norm) == 0.0


def test_non_finite_norms_follow_the_formula(ccr_mod):
    import torch
    work, norm = scratch(ccr_mod)
    with ccr_mod.Context(0) as c:
        for bad in (float("inf"), float("nan")):
            grads = [torch.ones(1000, device="cuda"), torch.ones(70, dtype=torch.bfloat16, device="cuda")]
            grads[1][3] = bad
            ccr_mod.ccr_grad_clip(c, grads, 1.0, work, norm)
            torch.cuda.synchronize()
            if bad != bad:
                assert norm.isnan().all() and all(bool(g.isnan().all()) for g in grads)
            else:
                assert float(norm) == bad and bool((grads[0] == 0).all()) and bool(grads[1][3].isnan())
        grads = [torch.ones(1000, device="cuda")]
        ccr_mod.ccr_grad_clip(c, grads, float("inf"), work, norm)
        assert close_norm(float(norm), math.sqrt(1000)) and bool((grads[0] == 1).all())
        ccr_mod.ccr_grad_clip(c, grads, 0.0, work, norm)
        assert bool((grads[0] == 0).all())
        for bad in (float("inf"), float("nan")):  # only measured
            grads = [torch.tensor([1.0, bad, 2.0], device="cuda")]
            ccr_mod.ccr_grad_clip(c, grads, float("inf"), work, norm)
            assert not bool(norm.isfinite()) and float(grads[0][0]) == 1.0 and float(grads[0][2]) == 2.0


def test_shared_tensors_count_twice_in_the_norm_only(ccr_mod):
    import torch
    work, norm = scratch(ccr_mod)
    x = torch.randn(5000, device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_grad_norm(c, [x, x, x[100:200]], work, norm)
        assert close_norm(float(norm), norm64([x, x, x[100:200]]))
        with pytest.raises(ccr_mod.CcrError, match="overlap"):
            ccr_mod.ccr_grad_clip(c, [x, x[100:200]], 1.0, work, norm)
        with pytest.raises(ccr_mod.CcrError, match="overlap"):
            ccr_mod.ccr_grad_clip(c, [x[:100]], 1.0, work, norm, out=[x[50:150]])


def test_refusals_write_nothing(ccr_mod):
    import ctypes

    import torch
    work, norm = scratch(ccr_mod)
    x = torch.ones(64, device="cuda")
    lib = ccr_mod._lib
    with ccr_mod.Context(0) as c:
        def raw(p=x.data_ptr(), count=64, dt=0, n=1, m=1.0, w=work.data_ptr(), o=norm.data_ptr()):
            return lib.ccr_grad_clip(c.handle, (ctypes.c_void_p * 1)(p), None, (ctypes.c_int64 * 1)(count),
                                     (ctypes.c_int32 * 1)(dt), n, m, w, o, None)

        for kw, word in [(dict(p=0), "NULL"), (dict(p=x.data_ptr() + 2), "aligned"), (dict(count=-1), "counts"),
                         (dict(count=1 << 39), "past the end"), (dict(dt=5), "dtypes"), (dict(n=-1), "n ="),
                         (dict(m=-1.0), "max_norm"), (dict(m=float("nan")), "max_norm"), (dict(w=0), "work"),
                         (dict(o=0), "norm"), (dict(o=x.data_ptr()), "overlap"),
                         (dict(w=norm.data_ptr()), "aligned" if norm.data_ptr() % 8 else "")]:
            st = raw(**kw)
            assert st != ccr_mod.CCR_OK and word in ccr_mod.ccr_last_error(), (kw, ccr_mod.ccr_last_error())
        with pytest.raises(TypeError):
            ccr_mod.ccr_grad_norm(c, [x.half()], work, norm)
        with pytest.raises(ValueError):
            ccr_mod.ccr_grad_norm(c, [torch.ones(8, 8, device="cuda").t()], work, norm)
        with pytest.raises(ValueError):
            ccr_mod.ccr_grad_norm(c, [x], work[:100], norm)
        torch.cuda.synchronize()
    assert bool((x == 1).all()) and norm.isnan().all()


def test_two_graphs_and_two_streams_with_their_own_work(ccr_mod):
    import torch
    sets = [grads_of([(300_001, "bf16", 1), (5000, "f32", 0)], seed=s, scale=s + 1.0) for s in range(2)]
    outs = [[torch.empty_like(x) for x in g] for g in sets]
    bufs = [scratch(ccr_mod) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    with ccr_mod.Context(0) as c:
        graphs = []
        for g, o, (w, n) in zip(sets, outs, bufs):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                ccr_mod.ccr_grad_clip(c, g, 1.0, w, n, out=o)
            graphs.append(graph)
        for step in range(3):
            for g in sets:
                for x in g:
                    x.copy_(torch.randn_like(x.float()).to(x.dtype))
            torch.cuda.synchronize()
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
            torch.cuda.synchronize()
            for g, o, (w, n) in zip(sets, outs, bufs):
                want = norm64(g)
                assert close_norm(float(n), want), f"replay {step}"
                got = [x.clone() for x in o]
                ccr_mod.ccr_grad_clip(c, g, 1.0, w, n, out=o)
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, o)), f"replay {step}"


@pytest.mark.parametrize("tiles", range(1, 14))
@pytest.mark.parametrize("where", ["in place", "apart"])
def test_one_launch_or_two(ccr_mod, tiles, where):
    """Norm and clipping of as many tiles of 16 KiB as one launch takes, and of one
    more, of one tensor, of one per tile, and of both types off a boundary."""
    import torch
    for sizes in ([(tiles * 4096, "f32", 0)], [(4096, "f32", 0)] * tiles, [(8192, "bf16", 0)] * tiles,
                  [(4096 - i % 3, "f32", i % 4) for i in range(tiles)],
                  [(8192 + i % 8, "bf16", (8 - i) % 8) for i in range(tiles)]):
        grads = grads_of(sizes, seed=tiles)
        w, n = Guarded((ccr_mod.CCR_GRAD_WORK,), torch.float64), Guarded((1,), torch.float32)
        with ccr_mod.Context(0) as c:
            ccr_mod.ccr_grad_norm(c, grads, w.t, n.t)
            torch.cuda.synchronize()
        assert close_norm(float(n.t), norm64(grads))
        n.t.fill_(float("nan"))
        outs = [Guarded((k,), tdtype(dt), offset_elements=off) for k, dt, off in sizes]
        check_clip(ccr_mod, grads, 0.5, w.t, n.t, out=None if where == "in place" else [o.t for o in outs])
        assert w.intact() and n.intact() and all(o.intact() for o in outs)
