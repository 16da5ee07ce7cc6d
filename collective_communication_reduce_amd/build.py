"""Build libccr.so (the C-ABI library) in place with hipcc for gfx950, and
_ccr_torch (the Python binding's marshalling of tensor lists) with g++ for the
interpreter and the torch that run this.

    python collective_communication_reduce_amd/build.py

Both are built in-tree next to this file so they travel with the source
tree; nothing is installed.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libccr.so")
MARSHAL = os.path.join(PKG, "_ccr_torch" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["ccr_api.cpp", "ccr_dma.cpp", "ccr_schedule.cpp", "ccr_kernels.hip", "ccr_ring.hip",
           "ccr_moe_kernels.hip", "ccr_experts.hip", "ccr_gate.hip", "ccr_grad.hip", "ccr_scratch.hip"]
# Per-source additions: the ring-hop kernels take their leading scalar
# arguments preloaded into registers (gfx950 kernel-argument preloading), so
# a workgroup's first scalar memory access is the load of its base addresses.
SOURCE_FLAGS = {"ccr_ring.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=16"],
                # assembled from a file that stays behind, which check_experts reads
                "ccr_experts.hip": ["-save-temps=obj"]}
ARCH = "gfx950"

# -packed-fp32-ops keeps the compiler from emitting packed fp32 arithmetic;
# denormals are kept (IEEE behaviour, no flush) and no FMA contraction is
# allowed, so fp32 sums are plain IEEE round-to-nearest-even adds.
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero", "-fno-fast-math",
    "-I" + os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found; the HIP library cannot be built")


def check_experts(asm: str) -> None:
    """Refuse an assembly of ccr_experts.hip whose hand-written instructions do
    not stand as they have to.

    The large tiles' matrix instructions are written in assembly, so the compiler
    does not wait for their results: between a loop's first product and the wait
    before the results are read it must not move an accumulator.  A load straight
    to LDS must not follow the write of its LDS place (m0) directly, and nothing
    else may write m0."""
    kernels = re.findall(r"^(_ZN3ccr\S*experts_big_kernel\S*):(.*?)s_endpgm", asm, re.S | re.M)
    if len(kernels) != 4:  # product, input gradient, weight gradient to fp32 and to bf16
        raise RuntimeError(f"ccr_experts.hip: {len(kernels)} kernels of large tiles, not 4")
    for name, body in kernels:
        loop = body[body.find("v_mfma"):]
        loop = loop[:loop.find("s_nop 15")]
        if loop.count("v_mfma") != 128 or "v_accvgpr" in loop or "scratch_" in loop:
            raise RuntimeError(f"ccr_experts.hip: an accumulator of {name} is moved between its products")
    lines = [x.split(";")[0].strip() for x in asm.splitlines()]
    lines = [x for x in lines if x and not x.startswith(".") and not x.endswith(":")]
    loads = [i for i, x in enumerate(lines) if x.startswith("global_load_lds")]
    if any(re.match(r"\w+ m0\b", lines[i - 1]) for i in loads):
        raise RuntimeError("ccr_experts.hip: a load to LDS directly behind the write of m0")
    if sum(bool(re.match(r"\w+ m0\b", x)) for x in lines) != len(loads):
        raise RuntimeError("ccr_experts.hip: m0 is written apart from the loads to LDS")


def build_marshal() -> str:
    """Compile _ccr_torch, the binding's marshalling of tensor lists: host code
    against torch's C++ headers, with torch's own C++ ABI."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include")]
    tmp = MARSHAL + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[a for i in inc for a in ("-isystem", i)], "-I" + sysconfig.get_paths()["include"],
           os.path.join(CSRC, "ccr_torch.cpp"), "-o", tmp, "-L" + os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on ccr_torch.cpp:\n{r.stdout}{r.stderr}")
    os.replace(tmp, MARSHAL)
    return MARSHAL


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *FLAGS, *SOURCE_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        noise = "is not a recognized feature for this target"
        err = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed on {src}:\n{err}")
        if src == "ccr_experts.hip":
            with open(os.path.join(BUILD, f"ccr_experts-hip-amdgcn-amd-amdhsa-{ARCH}.s")) as f:
                check_experts(f.read())
        if verbose and err.strip():
            print(err, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        marshal = ex.submit(build_marshal)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    # libhsa-runtime64 (SDMA engine copies): resolved at load time to the HSA
    # runtime already in the process (torch's), like libamdhip64.  The roctx
    # library marks each entry point for rocprofv3's marker trace.
    r = subprocess.run([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs,
                        "-L/opt/rocm/lib", "-lhsa-runtime64", "-lrocprofiler-sdk-roctx"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of libccr.so failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    marshal.result()  # the library stands without it
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
