"""The build of the 8-bit calls' marshalling: hipcc is its only compiler, the
module carries the interpreter's tag, and without the headers it is left out
with a warning, never kept from an earlier library."""

import os
import sysconfig

import pytest

import bit_weight_only_q4g64_amd as q4
from bit_weight_only_q4g64_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs the ROCm compilers")


@pytest.fixture
def place(tmp_path, monkeypatch):
    """The build writes into tmp_path, where an earlier untagged module lies."""
    out = tmp_path / os.path.basename(build.BINDING_OUT)
    monkeypatch.setattr(build, "BINDING_OUT", str(out))
    (tmp_path / "_a8.so").write_bytes(b"old")
    return tmp_path, out


def test_hipcc_is_the_only_compiler(place, monkeypatch):
    folder, out = place
    monkeypatch.setenv("PATH", "/opt/rocm/bin")
    monkeypatch.delenv("HIPCC", raising=False)
    assert build.build_binding() == str(out) and out.exists()
    assert [f.name for f in folder.iterdir()] == [out.name]


def test_left_out_without_the_headers(place, monkeypatch):
    folder, out = place
    out.write_bytes(b"old")
    monkeypatch.setattr(build, "binding_includes", lambda: [str(folder)])
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build_binding() is None
    assert list(folder.iterdir()) == []


def test_the_module_carries_the_interpreters_tag(monkeypatch):
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.basename(q4.BINDING_PATH) == "_a8" + suffix and q4.BINDING_PATH == build.BINDING_OUT
    assert sysconfig.get_config_var("SOABI") in suffix


def test_calls_name_what_is_missing(monkeypatch):
    monkeypatch.setattr(q4, "_bound", None)
    monkeypatch.setattr(q4, "BINDING_PATH", "/nonexistent/_a8.so")
    with pytest.raises(RuntimeError, match="headers"):
        q4.Act8.empty(1, 64, "cpu")
    q4.lib()  # the weight-only calls do not need it
