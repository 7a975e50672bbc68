"""The build where only the C library's tools are there: _torch_calls.so is left out with a warning."""
import os
import sys

import pytest

from tiled_gemm_f32_amd import build


@pytest.mark.parametrize("missing", ["torch", "g++", "headers"])
def test_torch_calls_are_optional(tmp_path, monkeypatch, missing):
    calls = tmp_path / "_torch_calls.so"
    calls.write_bytes(b"of other sources")
    monkeypatch.setattr(build, "CALLS_PATH", str(calls))
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif missing == "g++":
        monkeypatch.setenv("PATH", str(tmp_path))
    else:
        (tmp_path / "g++").write_text("#!/bin/sh\necho 'fatal error: Python.h: No such file or directory' >&2\nexit 1\n")
        os.chmod(tmp_path / "g++", 0o755)
        monkeypatch.setenv("PATH", f"{tmp_path}{os.pathsep}{os.environ['PATH']}")
    with pytest.warns(UserWarning, match="_torch_calls.so was not built"):
        assert build.build_torch_calls() is False
    assert not calls.exists()


def test_build_keeps_the_library_without_torch_calls(tmp_path, monkeypatch):
    """build() with every compiler run replaced: the library is linked and returned all the same."""
    monkeypatch.setattr(build, "CALLS_PATH", str(tmp_path / "_torch_calls.so"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libgemm.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "RESOURCE_FILE", str(tmp_path / "kernel_resources.json"))
    monkeypatch.setattr(build, "_compile", lambda src: (str(tmp_path / src), None))
    hipcc = tmp_path / "hipcc"
    hipcc.write_text("#!/bin/sh\nwhile [ \"$1\" != -o ]; do shift; done\necho linked > \"$2\"\n")
    os.chmod(hipcc, 0o755)
    monkeypatch.setattr(build, "HIPCC", str(hipcc))
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning):
        assert build.build() == str(tmp_path / "libgemm.so")
    assert (tmp_path / "libgemm.so").read_text() == "linked\n"
