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
    monkeypatch.setattr(_build, "TENSORS_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path / "out"))
    return _build


def modules(folder):
    return [f for f in os.listdir(folder) if f.startswith("_tensors") and f.endswith(".so")]


def test_without_torch(build, monkeypatch, capsys, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)          # (an import of it raises)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not modules(tmp_path) and "not built" in capsys.readouterr().err


def test_without_a_compiler(build, monkeypatch, capsys, tmp_path):
    monkeypatch.setenv("CXX", str(tmp_path / "no such program"))
    assert build.build() == build.LIB
    assert not modules(tmp_path) and "not built" in capsys.readouterr().err


def test_a_source_that_does_not_compile_is_tried_once(build, monkeypatch, capsys, tmp_path):
    runs, compiler = tmp_path / "runs", tmp_path / "compiler"
    compiler.write_text(f"#!/bin/sh\necho run >> '{runs}'\necho no such header >&2\nexit 1\n")
    compiler.chmod(0o755)
    monkeypatch.setenv("CXX", str(compiler))
    open(build.tensors_path(), "w").close()                  # of an earlier source
    os.utime(build.tensors_path(), (1, 1))
    for _ in range(3):
        assert build.build() == build.LIB
    assert runs.read_text() == "run\n" and "no such header" in capsys.readouterr().err
    assert not modules(tmp_path)
    build.build_tensors(force=True)
    assert runs.read_text() == "run\nrun\n"


def test_a_module_of_another_torch_or_python_is_not_opened(build, monkeypatch):
    """Its file carries the versions: for others there is none, the checks run in Python, and a build makes one."""
    import sysconfig
    import torch
    import int8_group_quantized_gb300 as dgq
    monkeypatch.setattr(build, "TENSORS_DIR", build.PKG)
    here = build.tensors_path()
    assert torch.__version__ in here and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(dgq, "_native_module", False)
    assert dgq._native() is not None
    others = set()
    for where, name, value in ((torch, "__version__", "2.12.0"), (torch.version, "git_version", "0" * 40),
                               (torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)):
        with monkeypatch.context() as m:
            m.setattr(where, name, value)
            others.add(build.tensors_path())
            m.setattr(dgq, "_native_module", False)
            assert dgq._native() is None
            x = torch.zeros(3, dtype=torch.int32)
            with pytest.raises(dgq.DGQError):                # (the checks in Python answer)
                dgq._operands("x", x, (x, torch.int32, (3,)))
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-313.so")
        others.add(build.tensors_path())
        m.setattr(dgq, "_native_module", False)
        assert dgq._native() is None
    assert len(others | {here}) == 5


def test_built_for_this_torch_and_found(build, monkeypatch, tmp_path):
    import int8_group_quantized_gb300 as dgq
    build.build()
    assert modules(tmp_path) == [os.path.basename(build.tensors_path())]
    monkeypatch.setattr(dgq, "_native_module", False)
    assert dgq._native().__file__ == build.tensors_path()
