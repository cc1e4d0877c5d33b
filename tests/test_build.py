"""What the build needs: nvcc alone for the C-ABI library; torch, its headers and
Python's for the module that takes tensors, and nothing of the library is lost
where that cannot be built."""
import ctypes
import os
import shutil

import pytest

from mla_decode_attention_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A library of one small source, built elsewhere."""
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("no nvcc")
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text('extern "C" int answer() { return 42; }\n')
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    return tmp_path


def answer(tree):
    return ctypes.CDLL(str(tree / build.LIB_NAME)).answer()


def test_the_library_is_built_without_torch(tree, monkeypatch):
    real = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    monkeypatch.setattr(build, "_compile_step", lambda: pytest.fail("torch is not there"))
    assert build.build() == str(tree / build.LIB_NAME)
    assert answer(tree) == 42 and not os.path.exists(tree / build._step_module())


def test_the_library_alone(tree, monkeypatch):
    monkeypatch.setattr(build, "_compile_step", lambda: pytest.fail("not asked for"))
    build.build(step=False)
    assert answer(tree) == 42


def test_a_module_that_does_not_build_is_an_error_that_leaves_the_library(tree, monkeypatch):
    def no_headers():
        raise RuntimeError("g++ failed on step_binding.cpp: Python.h not found")
    monkeypatch.setattr(build, "_compile_step", no_headers)
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert answer(tree) == 42


def test_the_module_is_built_where_it_alone_is_missing(tree, monkeypatch):
    """What the tests' session fixture calls."""
    made = []
    monkeypatch.setattr(build, "_compile_step", lambda: "step.o")
    monkeypatch.setattr(build, "_link_step", lambda obj: made.append(obj))
    assert build.build_step() == str(tree / build._step_module())
    assert made == ["step.o"] and not os.path.exists(tree / build.LIB_NAME)
