"""GPU parity of the norm and its gradients with 64-bit references where fp32 is
short of range or of digits."""
import math

import pytest

import rows8_helpers as r8
from gpu_helpers import say, torch_cuda
from operator_helpers import HALF, tdtype
from test_gpu_norm import U, check_q8, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ccr_mod():
    torch_cuda()
    import collective_communication_reduce_amd as ccr
    return ccr


@pytest.mark.parametrize("R,T,H,dt,rows", [(64, 262143, 8, "bf16", 16), (64, 262143, 264, "bf16", 8),
                                           (64, 65613, 1032, "bf16", 1), (1, 1 << 22, 1032, "bf16", 1),
                                           (64, 65613, 2060, "f32", 1), (64, 65613, 4104, "bf16", 1),
                                           (64, 16400, 16392, "bf16", 1)])
def test_weight_gradient_over_many_rows(ccr_mod, R, T, H, dt, rows):
    """Every row the same, with a product 0.49 units above a multiple of what a sum over
    the rows of one register (a workgroup has 1024 / R-th of a rank's, `rows` at a
    time) resolves, so that it would drift apart from the true one: chains of at
    most 128 additions each."""
    import torch
    d = tdtype(dt)
    need = (R + 1) * T * H * (2 if dt == "bf16" else 4)
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip(f"needs {need >> 30} GiB and 8 more")
    say(f"norm_bwd sums over {R} x {T} rows of {H} {dt}")
    unit = 2.0 ** (math.floor(math.log2(0.24 * T * R / 1024 / rows)) - 23)
    one = torch.ones(T, H, dtype=d, device="cuda")
    rstd = torch.full((T,), (math.floor(0.24 / unit) + 0.49) * unit, device="cuda")
    w = torch.ones(H, dtype=d, device="cuda")
    dx = [torch.empty_like(one) for _ in range(R)]
    dw = [torch.empty(H, device="cuda") for _ in range(R)]
    work = torch.empty(ccr_mod.ccr_rms_norm_work(R, T, H), device="cuda")
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_rms_norm_bwd(c, [one] * R, [one] * R, [w] * R, [rstd] * R, dx, dw, work)
        torch.cuda.synchronize()
    want = T * float(rstd[0].double())
    # 128 rows to a register, 128 of its sums, the 32 rows of a workgroup, the slots
    # by 64 threads, those by 2 and 16 more; and the products
    units = 128 + 128 + 32 + 16 + 2 + 16 + 2
    worst = max(float((v.double() - want).abs().max()) for v in dw) / (U * want)
    assert worst <= units, f"{worst} units"


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [32, 64, 104, 200, 1000, 2048, 8192, 16392])
def test_results_over_the_whole_range(ccr_mod, H, dt, add):
    """Rows of every magnitude without an eps, with zeros among their values: y and its
    8-bit rows, also where 1 / root is beyond fp32 or among its subnormal numbers."""
    import torch
    say(f"norm over the whole range H={H} {dt} add={add}")
    g = gen(H)
    d = tdtype(dt)
    sizes = [1.4e-45, 1e-43, 1e-40, 2.9e-39, 1e-38, 3e-20, 1.0, 7e19, 8e37, 1.7e38]
    x = torch.tensor(sizes, device="cuda")[:, None] * (2 * torch.rand(len(sizes), H, generator=g, device="cuda") - 1)
    x[:, 0] = torch.tensor(sizes, device="cuda")
    x[:, 3] = 0.0
    x[-1, 5] = 3.3e38
    x = x.to(d)
    if dt == "bf16":
        x[:2, 0] = 2.0 ** -133  # its smallest number
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(d)
    y = torch.empty_like(x)
    q = torch.empty(len(sizes), r8.row_bytes(H), dtype=torch.uint8, device="cuda")
    more = dict(residual=[torch.zeros_like(x)], h=[torch.empty_like(x)]) if add else {}
    with ccr_mod.Context(0) as c:
        ccr_mod.ccr_rms_norm(c, [x], [w], y=[y], q=[q], eps=0.0, **more)
        torch.cuda.synchronize()
    h = x.double()
    want = h * h.square().mean(1, keepdim=True).rsqrt() * w.double()
    # as for other rows: the root and two products, then the rounding; below the
    # smallest normal number three roundings of half the smallest step
    least = 2.0 ** -149 * 3 + (2.0 ** -134 if dt == "bf16" else 0)
    assert bool(((y.double() - want).abs() <= (HALF[dt] + 3.1 * U) * want.abs() + least).all())
    check_q8(q, want, 3.1 * U)
