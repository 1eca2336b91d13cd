"""The build (CPU): the library does not depend on its Python extension, and
the extension is rebuilt for another PyTorch or Python.  A one-kernel library
in a folder of its own stands for the real one."""
import os

import pytest

from w4a16_linear_layers_gb300 import build as qbuild
from w4a16_linear_layers_gb300 import qlin


@pytest.fixture
def small(tmp_path, monkeypatch):
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(qbuild, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(qbuild, "LIB_PATH", str(tmp_path / "libqlin.so"))
    monkeypatch.setattr(qbuild, "CALLS_PATH", str(tmp_path / "qlin_torch.so"))
    monkeypatch.setattr(qbuild, "_sources", lambda: [str(src)])
    return tmp_path


def fake_calls():
    """Writes what _build_calls leaves behind, without the compiler."""
    with open(qbuild.CALLS_PATH, "w"):
        pass
    with open(os.path.splitext(qbuild.CALLS_PATH)[0] + ".stamp", "w") as f:
        f.write(qbuild.calls_stamp())


def test_the_library_is_there_when_the_extension_fails(small, monkeypatch):
    def fails():
        raise FileNotFoundError("g++")
    monkeypatch.setattr(qbuild, "_build_calls", fails)
    with pytest.raises(RuntimeError, match="extension") as e:
        qbuild.build()
    assert isinstance(e.value.__cause__, FileNotFoundError)
    assert os.path.exists(qbuild.LIB_PATH)
    assert not qbuild.up_to_date()
    before = os.path.getmtime(qbuild.LIB_PATH)
    monkeypatch.setattr(qbuild, "_build_calls", fake_calls)
    assert qbuild.build() == qbuild.LIB_PATH
    assert qbuild.up_to_date() and os.path.getmtime(qbuild.LIB_PATH) == before


def test_no_extension_without_pytorch(small, monkeypatch):
    def fails():
        raise AssertionError("called")
    monkeypatch.setattr(qbuild, "_build_calls", fails)
    monkeypatch.setattr(qbuild, "calls_stamp", lambda: None)
    assert qbuild.build() == qbuild.LIB_PATH and os.path.exists(qbuild.LIB_PATH)
    assert qbuild.up_to_date()


def test_another_pytorch_or_python_rebuilds_the_extension(small, monkeypatch):
    built = []

    def calls():
        built.append(qbuild.calls_stamp())
        fake_calls()
    monkeypatch.setattr(qbuild, "_build_calls", calls)
    qbuild.build()
    here = qbuild.calls_stamp()
    assert "torch" in here and built == [here] and qbuild.up_to_date()
    qbuild.build()
    assert built == [here]
    monkeypatch.setattr(qbuild, "calls_stamp", lambda: "torch 99, python 4")
    assert not qbuild.up_to_date()
    qbuild.build()
    assert built == [here, "torch 99, python 4"] and qbuild.up_to_date()
    assert qbuild.calls_built_for() == "torch 99, python 4"


def test_an_extension_for_something_else_is_not_loaded(monkeypatch):
    qbuild.build()
    qlin.load()
    monkeypatch.setattr(qlin, "_torch_calls", None)
    monkeypatch.setattr(qbuild, "calls_stamp", lambda: "torch 99, python 4")
    with pytest.raises(qlin.QlinError, match="torch 99"):
        qlin._calls()


def test_a_pytorch_that_is_not_installed(monkeypatch):
    """One that is only in the path has no metadata."""
    def none(name):
        raise qbuild.importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(qbuild.importlib.metadata, "version", none)
    import torch
    assert torch.__version__ in qbuild.calls_stamp()


def test_the_extension_loads():
    qbuild.build()
    assert qbuild.calls_built_for() == qbuild.calls_stamp()
    for name in ("add_rmsnorm", "gemm_ch", "adjust_logits"):
        assert callable(getattr(qlin._calls(), name))
