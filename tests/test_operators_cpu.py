"""Host-side refusals of the experts' products, the gated sum and the gradient
calls: what the binding and the C entries turn away before any device is
touched.  No GPU is used."""
import os
import re
import subprocess
import sys
import sysconfig
import types

import numpy as np
import pytest
import torch

import collective_communication_reduce_amd as ccr
from collective_communication_reduce_amd import build as ccr_build

CTX = types.SimpleNamespace(device=0, handle=None)
BF16 = torch.bfloat16


def test_a_null_context_is_refused():
    n = np.zeros((1, 2), np.int64).ctypes.data
    lib = ccr._lib
    calls = [lib.ccr_moe_experts(None, None, None, n, 1, 2, 8, 8, 1, None, None),
             lib.ccr_moe_experts_dgrad(None, None, None, n, 1, 2, 8, 8, 1, None, None),
             lib.ccr_moe_experts_wgrad(None, None, None, n, 1, 2, 8, 8, 1, 0, 0, None, None),
             lib.ccr_moe_gate_sum(None, None, None, None, 1, 1, 2, 1, 8, 1, 0, None, None),
             lib.ccr_moe_gate_sum_bwd(None, None, None, None, None, 1, 1, 2, 1, 8, 1, 0, None, None, None),
             lib.ccr_grad_norm(None, None, None, None, 0, None, None, None),
             lib.ccr_grad_clip(None, None, None, None, None, 0, 1.0, None, None, None)]
    assert calls == [ccr.CCR_ERR_INVALID_ARG] * len(calls)
    assert "ctx" in ccr.ccr_last_error()
    assert lib.ccr_moe_experts_wgrad(None, None, None, n, 1, 2, 8, 8, 1, 0, 2, None, None) == \
        ccr.CCR_ERR_INVALID_ARG
    assert "accumulate" in ccr.ccr_last_error()


def test_host_tensors_are_refused():
    x, w, y = torch.ones(3, 16), torch.ones(2, 8, 16), torch.ones(3, 8)
    ecnt = [[1, 2]]
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_moe_experts(CTX, [x], [w], ecnt, [y])
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_moe_experts_dgrad(CTX, [y], [w], ecnt, [x])
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_moe_experts_wgrad(CTX, [x], [y], ecnt, [w])
    rows, logits, topk = torch.ones(3, 2, 8), torch.ones(3, 4), torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_moe_gate_sum(CTX, [rows], [logits], [topk], [torch.ones(3, 8)])
    with pytest.raises(ValueError, match="device tensor"):
        ccr.ccr_grad_norm(CTX, [x], None, None)


def test_types_and_shapes_are_refused():
    x, w, y = torch.ones(3, 16, dtype=BF16), torch.ones(2, 8, 16, dtype=BF16), torch.ones(3, 8, dtype=BF16)
    with pytest.raises(TypeError):  # operands of two types
        ccr.ccr_moe_experts(CTX, [x.float()], [w], [[1, 2]], [y])
    with pytest.raises(TypeError):
        ccr.ccr_moe_experts(CTX, [x.half()], [w.half()], [[1, 2]], [y.half()])
    with pytest.raises(ValueError, match="ecnt"):
        ccr.ccr_moe_experts(CTX, [x], [w], [1, 2], [y])
    with pytest.raises(ValueError, match="ecnt"):
        ccr.ccr_moe_experts(CTX, [x] * 2, [w] * 2, [[1, 2, 0], [0, 0, 0]], [y] * 2)
    with pytest.raises(ValueError, match="buffers"):
        ccr.ccr_moe_experts(CTX, [x, x], [w], [[1, 2]], [y])
    with pytest.raises(TypeError):
        ccr.ccr_grad_clip(CTX, [torch.ones(4).double()], 1.0, None, None)
    with pytest.raises(ValueError, match="norm"):
        ccr.ccr_moe_gate_sum(CTX, [], [], [], [], norm="some")


def test_work_constant_matches_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(ccr.__file__)))
    text = open(os.path.join(root, "include", "ccr.h")).read()
    assert int(re.search(r"#define CCR_GRAD_WORK (\d+)", text).group(1)) == ccr.CCR_GRAD_WORK


def test_no_accumulator_is_copied_between_products(tmp_path):
    # The large tiles' products are written in assembly, so the compiler does not
    # wait for them: between a loop's first product and the wait before the results
    # are read it must not move an accumulator.
    asm = tmp_path / "experts.s"
    subprocess.run([ccr_build.hipcc(), *ccr_build.FLAGS, "-S", "--offload-device-only",
                    os.path.join(ccr_build.CSRC, "ccr_experts.hip"), "-o", str(asm)],
                   check=True, capture_output=True)
    text = asm.read_text()
    kernels = re.findall(r"^(_ZN3ccr\S*experts_big_kernel\S*):(.*?)s_endpgm", text, re.S | re.M)
    assert len(kernels) == 4  # product, input gradient, weight gradient to fp32 and to bf16
    for name, body in kernels:
        loop = body[body.index("v_mfma"):]
        loop = loop[:loop.index("s_nop 15")]
        assert loop.count("v_mfma") == 128, name
        assert "v_accvgpr" not in loop and "scratch_" not in loop, name


@pytest.fixture(scope="module")
def experts_asm(tmp_path_factory):
    asm = tmp_path_factory.mktemp("asm") / "experts.s"
    subprocess.run([ccr_build.hipcc(), *ccr_build.FLAGS, "-S", "--offload-device-only",
                    os.path.join(ccr_build.CSRC, "ccr_experts.hip"), "-o", str(asm)],
                   check=True, capture_output=True)
    return asm.read_text()


def test_no_load_to_lds_follows_the_write_of_m0_directly(experts_asm):
    # m0 holds the LDS place of a load that goes straight there; the load needs a
    # wait state between the write and itself, or it may take the place before.
    lines = [x.split(";")[0].strip() for x in experts_asm.splitlines()]
    lines = [x for x in lines if x and not x.startswith(".") and not x.endswith(":")]
    loads = [i for i, x in enumerate(lines) if x.startswith("global_load_lds")]
    assert len(loads) > 64
    bare = [lines[i - 1:i + 1] for i in loads if re.match(r"s_\w+ m0\b", lines[i - 1])]
    assert not bare, f"{len(bare)} of {len(loads)}, first {bare[0]}"
    # nothing but these loads writes m0
    assert sum(bool(re.match(r"\w+ m0\b", x)) for x in lines) == len(loads)


def test_the_build_refuses_moved_accumulators_and_bare_loads(experts_asm):
    ccr_build.check_experts(experts_asm)
    at = experts_asm.index("v_mfma", experts_asm.index("experts_big_kernel"))
    end = experts_asm.index("\n", at) + 1
    for planted in ("\tv_accvgpr_read_b32 v0, a0\n", "\tscratch_store_dword off, v0, s0\n"):
        with pytest.raises(RuntimeError, match="moved"):
            ccr_build.check_experts(experts_asm[:end] + planted + experts_asm[end:])
    with pytest.raises(RuntimeError, match="m0"):
        ccr_build.check_experts(experts_asm[:end] + "\ts_mov_b32 m0, s0\n" + experts_asm[end:])
    load = re.search(r"\ts_add_u32 m0, .*\n(\ts_nop 0\n)\tglobal_load_lds", experts_asm)
    with pytest.raises(RuntimeError, match="m0"):
        ccr_build.check_experts(experts_asm[:load.start(1)] + experts_asm[load.end(1):])
    with pytest.raises(RuntimeError, match="kernels"):
        ccr_build.check_experts("")


def test_the_build_checks_what_it_links(monkeypatch, tmp_path):
    done = []
    monkeypatch.setattr(ccr_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(ccr_build, "build_marshal", lambda: "")
    monkeypatch.setattr(ccr_build.subprocess, "run", lambda cmd, **k: done.append(cmd) or types.SimpleNamespace(
        returncode=0, stdout="", stderr=""))
    (tmp_path / f"ccr_experts-hip-amdgcn-amd-amdhsa-{ccr_build.ARCH}.s").write_text("s_endpgm")
    with pytest.raises(RuntimeError, match="large tiles"):
        ccr_build.build()
    assert not any("-shared" in cmd for cmd in done)  # nothing was linked
    # the checked file is the one that the object is assembled from
    assert any("-save-temps=obj" in cmd and cmd[-1] == str(tmp_path / "ccr_experts.o") for cmd in done)


def test_rows_beyond_the_counted_ones_are_taken_where_they_are_left_alone():
    x = torch.ones(5, 2)
    for shape, room, word in [((4, 2), True, "device tensor"), ((5, 2), True, "device tensor"),
                              ((6, 2), True, "shape"), ((4, 2), False, "shape"), ((5, 2), False, "device tensor"),
                              ((5, 1), True, "shape"), ((5,), True, "shape"), ((5, 2, 1), True, "shape")]:
        with pytest.raises(ValueError, match=word):
            ccr._buffers(CTX, [x], torch.float32, [shape], "x", room)


def test_the_collectives_do_without_the_marshalling_module(tmp_path):
    """Without the compiled module the package loads and its other calls work; the
    calls that need it say what is missing."""
    pkg = tmp_path / "collective_communication_reduce_amd"
    pkg.mkdir()
    home = os.path.dirname(os.path.abspath(ccr.__file__))
    for name in ("__init__.py", "libccr.so"):
        os.symlink(os.path.join(home, name), pkg / name)
    code = """
import sys, types
import torch
import collective_communication_reduce_amd as ccr
assert ccr.__file__.startswith(sys.argv[1]), ccr.__file__
print(ccr.ccr_version(), ccr.ccr_config_default().slices, "_ccr_torch" in "".join(sys.modules))
try:
    ccr.ccr_grad_norm(types.SimpleNamespace(device=0, handle=None), [], None, None)
except ImportError as e:
    print("refused:", e)
"""
    env = dict(os.environ, PYTHONPATH=str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code, str(tmp_path)], capture_output=True, text=True, env=env,
                       cwd=tmp_path)
    assert r.returncode == 0, r.stderr
    first, second = r.stdout.splitlines()
    assert first == f"{ccr.ccr_version()} {ccr.ccr_config_default().slices} False"
    assert second.startswith("refused:") and "_ccr_torch" in second and "build.py" in second


@pytest.mark.parametrize("abi", [False, True])
def test_the_marshalling_module_is_built_for_this_torch_and_python(monkeypatch, tmp_path, abi):
    done = []
    monkeypatch.setattr(ccr_build, "MARSHAL", str(tmp_path / os.path.basename(ccr_build.MARSHAL)))
    monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: abi)
    monkeypatch.setattr(ccr_build.subprocess, "run", lambda cmd, **k: done.append(cmd) or
                        open(cmd[cmd.index("-o") + 1], "w").close() or types.SimpleNamespace(returncode=0))
    assert ccr_build.build_marshal().endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert f"-D_GLIBCXX_USE_CXX11_ABI={int(abi)}" in done[0]
