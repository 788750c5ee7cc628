"""The library is built where the Python entry of the decoder-layer operators cannot be; both are rebuilt when they
have to be.  On small sources of their own."""
import os
import sysconfig

import pytest
import torch

from w4a4_quantized_gemm_gb300 import build as wbuild

CU = 'extern "C" int answer() { return 42; }\n'
CPP = '#include <Python.h>\nextern "C" int answer();\nextern "C" int ask() { return answer(); }\n'


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "a.cu").write_text(CU)
    (csrc / "binding.cpp").write_text(CPP)
    for name, value in dict(HERE=str(tmp_path), ROOT=str(tmp_path), CSRC=str(csrc), BUILD=str(tmp_path / "_build"),
                            LIB=str(tmp_path / "libw4a4.so"), BINDING_SRC=str(csrc / "binding.cpp"),
                            BINDING=str(tmp_path / "_binding.so")).items():
        monkeypatch.setattr(wbuild, name, value)
    return tmp_path


def no_headers(monkeypatch, tmp_path):
    paths = {**sysconfig.get_paths(), "include": str(tmp_path / "nothing")}
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)


def test_library_without_the_binding(tree, monkeypatch):
    """No Python.h: the C library, which needs none, is built, and a warning says what is missing."""
    with monkeypatch.context() as m:
        no_headers(m, tree)
        (tree / "_binding.so").write_text("of an earlier build")
        os.utime(tree / "_binding.so", (1, 1))
        with pytest.warns(RuntimeWarning, match="binding"):
            assert wbuild.build() == str(tree / "libw4a4.so")
        assert os.path.exists(tree / "libw4a4.so") and not os.path.exists(tree / "_binding.so")
        assert not wbuild.up_to_date()
    made = os.path.getmtime(tree / "libw4a4.so")
    wbuild.build()  # the headers are there again: the binding alone
    assert os.path.exists(tree / "_binding.so") and os.path.getmtime(tree / "libw4a4.so") == made
    assert wbuild.up_to_date()


def test_an_error_in_the_library_stays_an_error(tree):
    (tree / "csrc" / "a.cu").write_text("not C++\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        wbuild.build()


def test_binding_is_rebuilt_for_another_torch_or_python(tree, monkeypatch):
    wbuild.build()
    assert wbuild.up_to_date()
    made = os.path.getmtime(tree / "libw4a4.so")
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert not wbuild.up_to_date()
    wbuild.build()
    assert wbuild.up_to_date() and os.path.getmtime(tree / "libw4a4.so") == made
