"""Build the q4g64 HIP library in-tree for gfx950.

    python -m bit_weight_only_q4g64_amd.build

compiles the two translation units ``csrc/api.hip`` (the weight-only matmuls)
and ``csrc/a8.hip`` (the 8-bit activation path) side by side and links them into
``bit_weight_only_q4g64_amd/libq4g64.so``, then compiles the C++ marshalling of
the 8-bit calls (``csrc/a8_binding.cpp``, host code only) into an extension
module of this interpreter beside it (``_a8.cpython-....so``). hipcc compiles
both. The marshalling also needs Python's and torch's headers; where they are
missing, the build warns and leaves it out, and only the 8-bit calls are
unavailable. Strict IEEE float32: no fast-math and no floating-point
contraction (every fused multiply-add in the kernels is an explicit fma), no
packed-fp32 instructions, and matrix-core results kept in ordinary vector
registers.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRCS = [os.path.join(HERE, "csrc", name) for name in ("api.hip", "a8.hip")]
OUT = os.path.join(HERE, "libq4g64.so")
BINDING_SRC = os.path.join(HERE, "csrc", "a8_binding.cpp")
BINDING_OUT = os.path.join(HERE, "_a8" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_HEADERS = ("Python.h", "ATen/ATen.h", "ATen/hip/EmptyTensor.h", "torch/csrc/autograd/python_variable.h")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-Xclang",
    "-target-feature",
    "-Xclang",
    "-packed-fp32-ops",
    # matrix-core results in ordinary vector registers rather than the
    # accumulation registers: the same instructions (so the same bits), minus
    # the copies between the two files before each fold; measured 1.2x on
    # the short-window GEMM, no change on the others
    "-mllvm",
    "-amdgpu-mfma-vgpr-form",
    "-Wall",
    "-Wno-unused-result",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the q4g64 library)")


def build(verbose: bool = False) -> str:
    """Compile the library (always recompiles) and return its path."""
    tmp = OUT + ".tmp"
    noise = "is not a recognized feature for this target"
    objs = [src[: -len(".hip")] + ".o" for src in SRCS]
    flags = [f for f in FLAGS if f != "-shared"]
    cmds = [[hipcc(), *flags, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj] for src, obj in zip(SRCS, objs)]
    runs = [(cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)) for cmd in cmds]
    done = [(cmd, *run.communicate(), run.returncode) for cmd, run in runs]
    link = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    for cmd, _, stderr, rc in done:
        err = "\n".join(line for line in stderr.splitlines() if noise not in line)
        if rc != 0:
            raise RuntimeError(f"hipcc failed ({rc}):\n{' '.join(cmd)}\n{err}")
        if verbose and err.strip():
            print(err, file=sys.stderr)
    res = subprocess.run(link, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{' '.join(link)}\n{res.stderr}")
    os.replace(tmp, OUT)
    build_binding()
    return OUT


def binding_includes() -> list:
    """Folders of the headers that the marshalling is compiled against: torch's and this interpreter's."""
    import torch

    root = os.path.join(os.path.dirname(torch.__file__), "include")
    return [root, os.path.join(root, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"]]


def build_binding() -> str | None:
    """Compile the C++ marshalling against this interpreter's torch, with its ABI, and return its path; None (and a
    warning) where the headers are missing. What was there before goes first: it is of another library."""
    import torch

    for old in (BINDING_OUT, os.path.join(os.path.dirname(BINDING_OUT), "_a8.so")):
        if os.path.exists(old):
            os.remove(old)
    inc = binding_includes()
    missing = [h for h in BINDING_HEADERS if not any(os.path.exists(os.path.join(d, h)) for d in inc)]
    if missing:
        warnings.warn(f"the 8-bit calls are left out: no {', '.join(missing)} in {', '.join(inc)}")
        return None
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_OUT + ".tmp"
    cmd = [hipcc(), "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in (*inc, os.path.join(rocm, "include"))),
           BINDING_SRC, "-o", tmp, f"-L{HERE}", "-l:libq4g64.so", f"-L{libs}", "-ltorch", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python",
           "-lc10", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{' '.join(cmd)}\n{res.stderr}")
    os.replace(tmp, BINDING_OUT)
    return BINDING_OUT


if __name__ == "__main__":
    print(build(verbose=True))
