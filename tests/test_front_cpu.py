"""Host-side refusals of the norm, the router, 8-bit rows and the products on
them, and what the build asks of the products' assembly.  No GPU is used."""
import os
import re
import subprocess
import types

import numpy as np
import pytest
import torch

import collective_communication_reduce_amd as ccr
import rows8_helpers as r8
from collective_communication_reduce_amd import build as ccr_build

CTX = types.SimpleNamespace(device=0, handle=None)
BF16 = torch.bfloat16


def test_a_null_context_is_refused():
    n = np.zeros((1, 2), np.int64).ctypes.data
    lib, how = ccr._lib, ccr.ccr_route_t(0, 1, 1, 1, 1, 1.0)
    calls = [lib.ccr_rms_norm(None, None, None, None, 1, 1, 8, 1, 1, 1e-6, None, None, None, None, None),
             lib.ccr_rms_norm_bwd(None, None, None, None, None, None, 1, 1, 8, 1, 1, 0, None, None, None, None),
             lib.ccr_quantize_rows(None, None, None, 1, 8, 1, None, None),
             lib.ccr_dequantize_rows(None, None, None, 1, 8, 1, None, None),
             lib.ccr_moe_experts_q8(None, None, None, n, 1, 2, 8, 8, None, None),
             lib.ccr_moe_route(None, None, None, 1, 1, 2, 1, how, None, None, None, None, None, None),
             lib.ccr_moe_route_bwd(None, None, None, None, None, 1, 1, 2, 1, 0, 1, 1.0, None, None)]
    assert calls == [ccr.CCR_ERR_INVALID_ARG] * len(calls)
    assert "ctx" in ccr.ccr_last_error()


def test_sizes():
    for H in [1, 8, 31, 32, 127, 128, 129, 2048, 4096, 4104, 1 << 20]:
        assert ccr.ccr_q8_row_bytes(H) == r8.row_bytes(H)
    assert [ccr.ccr_q8_row_bytes(H) for H in (-8, 0, (1 << 20) + 1)] == [0, 0, 0]
    # a slot of H values per workgroup, at most 1024 workgroups, one per row
    assert ccr.ccr_rms_norm_work(1, 1, 64) >= 64
    assert 8 * 2048 <= ccr.ccr_rms_norm_work(8, 4096, 2048) <= 1024 * 2048
    assert [ccr.ccr_rms_norm_work(*x) for x in ((0, 1, 8), (65, 1, 8), (1, 0, 8), (1, 1, 0))] == [0] * 4
    assert ccr.ccr_moe_route_work(1, 1, 64) >= 2 * 64
    assert [ccr.ccr_moe_route_work(*x) for x in ((0, 1, 8), (65, 1, 8), (1, 0, 8), (1, 1, 1025))] == [0] * 4


def test_host_tensors_are_refused():
    x, w = torch.ones(3, 16), torch.ones(16)
    q = torch.zeros(3, r8.row_bytes(16), dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_rms_norm(CTX, [x], [w], y=[x])
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_rms_norm_bwd(CTX, [x], [x], [w], [x[:, 0]], [x], [w], w)
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_quantize_rows(CTX, [x], [q])
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_dequantize_rows(CTX, [q], [x])
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_moe_experts_q8(CTX, [q], [q[None]], [[3]], 16, [x.to(BF16)])
    top = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_moe_route(CTX, [x], [top], [torch.ones(3, 2)])
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_moe_route_bwd(CTX, [x], [top], [torch.ones(3, 2)], [x])


def test_types_shapes_and_words_are_refused():
    x, w = torch.ones(3, 16), torch.ones(16)
    with pytest.raises(ValueError, match="score"):
        ccr.ccr_moe_route(CTX, [x], [x], [x], score="relu")
    with pytest.raises(ValueError, match="score"):
        ccr.ccr_moe_route_bwd(CTX, [x], [x], [x], [x], score="relu")
    with pytest.raises(ValueError, match="buffers"):
        ccr._buffers(CTX, [x], x.dtype, [], "x")
    with pytest.raises(ValueError, match="work"):
        ccr._work(CTX, None, 5)
    assert ccr._work(CTX, None, 0) is None
    with pytest.raises(ValueError, match="shape"):
        ccr._work(CTX, x.view(-1), 49)


def test_the_format_of_the_tests_is_the_documented_one():
    """e4m3 as torch has it, scales the smallest that hold their block."""
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(b), np.isnan(r8.VALUES)) and np.array_equal(b[~np.isnan(b)], r8.VALUES[~np.isnan(b)])
    rng = np.random.default_rng(1)
    x = rng.normal(size=(50, 100)) * 10.0 ** rng.integers(-30, 30, size=(50, 1))
    rows = r8.pack(x)
    v, s = r8.unpack(rows, 100)
    top = np.zeros((50, 128))
    top[:, :100] = np.abs(x)
    top = top.reshape(50, 4, 32).max(axis=2)
    assert (448 * np.ldexp(1.0, s - 127) >= top).all() and ((224 * np.ldexp(1.0, s - 127) < top) | (s == 0)).all()
    assert np.array_equal(r8.unpack(r8.pack(v), 100)[0], v)  # values on the grid stay
    x = x.astype(np.float32)  # torch rounds from fp32
    rows, s = r8.pack(x), r8.unpack(r8.pack(x), 100)[1]
    t = torch.from_numpy(np.ldexp(x.astype(np.float64), 127 - np.repeat(s, 32, axis=1)[:, :100]))
    assert np.array_equal(t.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy(), rows[:, :100])


@pytest.fixture(scope="module")
def experts8_asm(tmp_path_factory):
    asm = tmp_path_factory.mktemp("asm") / "experts8.s"
    subprocess.run([ccr_build.hipcc(), *ccr_build.FLAGS, "-S", "--offload-device-only",
                    os.path.join(ccr_build.CSRC, "ccr_experts8.hip"), "-o", str(asm)],
                   check=True, capture_output=True)
    return asm.read_text()


def test_the_build_refuses_moved_accumulators_and_bare_loads(experts8_asm):
    ccr_build.check_experts8(experts8_asm)
    at = experts8_asm.index("v_mfma", experts8_asm.index("experts8_big_kernel"))
    end = experts8_asm.index("\n", at) + 1
    for planted in ("\tv_accvgpr_read_b32 v0, a0\n", "\tscratch_store_dword off, v0, s0\n"):
        with pytest.raises(RuntimeError, match="moved"):
            ccr_build.check_experts8(experts8_asm[:end] + planted + experts8_asm[end:])
    with pytest.raises(RuntimeError, match="m0"):
        ccr_build.check_experts8(experts8_asm[:end] + "\ts_mov_b32 m0, s0\n" + experts8_asm[end:])
    load = re.search(r"\ts_add_u32 m0, .*\n(\ts_nop 0\n)\t(?:global_load_lds|buffer_load)", experts8_asm)
    with pytest.raises(RuntimeError, match="m0"):
        ccr_build.check_experts8(experts8_asm[:load.start(1)] + experts8_asm[load.end(1):])
    with pytest.raises(RuntimeError, match="kernels"):
        ccr_build.check_experts8("")
    assert set(ccr_build.CHECKS) <= set(ccr_build.SOURCES)
    assert all("-save-temps=obj" in ccr_build.SOURCE_FLAGS[s] for s in ccr_build.CHECKS)
