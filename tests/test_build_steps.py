"""libbl.so needs nvcc only: what keeps the tensor binding from being built does not keep the C library from it."""
import importlib.util
import os

import pytest

from matrix_dense_linear_spd_gb300 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The objects of an up-to-date build, linked into a folder of the test's."""
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    build.build()
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libbl.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_torch_binding.so"))
    return tmp_path


def test_both_are_built(elsewhere):
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)


def test_a_binding_that_does_not_compile_leaves_the_library(elsewhere, monkeypatch):
    def broken():
        raise RuntimeError("no headers")
    monkeypatch.setattr(build, "_compile_binding", broken)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_without_torch_there_is_a_library_and_no_binding(elsewhere, monkeypatch, capsys):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "torch is not installed" in capsys.readouterr().err
