"""What the 8-bit activation calls launch, asked without a GPU: the host code
of a8.hip, compiled host-only and linked against a recorder in the HIP
runtime's place (tests/host/launch_record.cpp)."""

import atexit
import functools
import os
import pathlib
import re
import shutil
import subprocess
import tempfile
from typing import NamedTuple

ROOT = pathlib.Path(__file__).resolve().parents[1]
CSRC = ROOT / "bit_weight_only_q4g64_amd" / "csrc"
DRIVER = ROOT / "tests" / "host" / "launch_record.cpp"
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"

available = os.path.exists(HIPCC) and os.path.exists(CLANG)


class Launch(NamedTuple):
    kernel: str  # the demangled name with its template arguments
    workgroups: int
    lanes: int


class Call(NamedTuple):
    status: int
    work_bytes: int
    launches: tuple


@functools.lru_cache(None)
def _program() -> pathlib.Path:
    """The recorder, built once per process."""
    tmp = pathlib.Path(tempfile.mkdtemp(prefix="launch_record_"))
    atexit.register(shutil.rmtree, tmp, True)
    (tmp / "empty.hipfb").write_bytes(b"")  # no device code
    for cmd in (
        [HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-Xclang", "-fcuda-include-gpubinary",
         "-Xclang", tmp / "empty.hipfb", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", ROOT / "include", "-c", CSRC / "a8.hip", "-o", tmp / "a8.o"],
        [CLANG, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", ROOT / "include", "-I", "/opt/rocm/include", DRIVER, tmp / "a8.o",
         "-o", tmp / "launch_record"],
    ):
        r = subprocess.run([str(c) for c in cmd], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-4000:]
    return tmp / "launch_record"


def record(calls) -> list:
    """The Call of every ("quant" | "norm" | "product" | "pair" | "swiglu", M, ..., K[, "f32" | "bf16"])."""
    text = "".join(" ".join(str(v) for v in c) + "\n" for c in calls)
    r = subprocess.run([str(_program())], input=text, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    out = []
    for line in r.stdout.splitlines():
        head, *rest = line.split("|")
        status, work = head.split()
        launches = tuple(Launch(re.sub(r"^void |\(q4::.*$", "", rest[i]), int(rest[i + 1]), int(rest[i + 2])) for i in range(0, len(rest), 3))
        out.append(Call(int(status), int(work), launches))
    return out
