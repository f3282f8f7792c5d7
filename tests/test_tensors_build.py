"""The native module with the binding's checks is an extra: the library builds without torch and without a C++
compiler, and what cannot be built is left out.  CPU only."""
import os
import sys

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build, with the module's place somewhere else."""
    from int8_group_quantized_gb300 import _build
    _build.build()
    monkeypatch.setattr(_build, "TENSORS", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path / "out"))
    return _build


def test_without_torch(build, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)          # (an import of it raises)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.TENSORS) and "not built" in capsys.readouterr().err


def test_without_a_compiler(build, monkeypatch, capsys, tmp_path):
    monkeypatch.setenv("CXX", str(tmp_path / "no such program"))
    assert build.build() == build.LIB
    assert not os.path.exists(build.TENSORS) and "not built" in capsys.readouterr().err


def test_a_source_that_does_not_compile_is_tried_once(build, monkeypatch, capsys, tmp_path):
    runs, compiler = tmp_path / "runs", tmp_path / "compiler"
    compiler.write_text(f"#!/bin/sh\necho run >> '{runs}'\necho no such header >&2\nexit 1\n")
    compiler.chmod(0o755)
    monkeypatch.setenv("CXX", str(compiler))
    open(build.TENSORS, "w").close()                         # of an earlier source
    os.utime(build.TENSORS, (1, 1))
    for _ in range(3):
        assert build.build() == build.LIB
    assert runs.read_text() == "run\n" and "no such header" in capsys.readouterr().err
    assert not os.path.exists(build.TENSORS)
    build.build_tensors(force=True)
    assert runs.read_text() == "run\nrun\n"
