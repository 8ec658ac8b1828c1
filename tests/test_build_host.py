"""What build() makes, and for which Python and torch: the step calls' module
reads tensors by the headers it was compiled with."""

import os

import pytest
import torch

import paged_split_kv_02_gb300 as pd
from paged_split_kv_02_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()


def test_the_module_is_named_after_its_python_and_torch():
    assert torch.__version__ in os.path.basename(_build.BIND) and os.path.exists(_build.BIND)
    assert _build.bind_path(torch_version="2.0.0") != _build.BIND != _build.bind_path(python="cpython-311")
    assert _build.up_to_date() and _build.bind_up_to_date()


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(pd, "_bind", None)
    monkeypatch.setattr(_build, "BIND", _build.bind_path(torch_version="2.0.0"))
    with pytest.raises(RuntimeError, match="torch2.0.0.so is missing"):
        pd._step("attn_sinks")


def test_another_torch_gets_its_own_module_and_the_library_stays(monkeypatch, tmp_path):
    made = []
    monkeypatch.setattr(_build, "BIND", str(tmp_path / "_bind.other.so"))
    monkeypatch.setattr(_build, "_build_lib", lambda *a: made.append("library"))
    monkeypatch.setattr(_build, "_build_bind", lambda *a: made.append("module"))
    assert not _build.bind_up_to_date()
    assert _build.build() == _build.LIB and made == ["module"]
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "other.so"))
    made.clear()
    _build.build()
    assert sorted(made) == ["library", "module"]


def test_a_machine_that_cannot_compile_the_module_still_has_the_library(monkeypatch, tmp_path):
    made = []
    monkeypatch.setattr(pd, "_bind", None)
    monkeypatch.setattr(_build, "BIND", str(tmp_path / "_bind.other.so"))
    monkeypatch.setattr(_build, "_build_lib", lambda *a: made.append("library"))
    assert _build.bind_missing() == ""
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert _build.bind_missing() == str(tmp_path / "Python.h")
    with pytest.warns(UserWarning, match="Python.h is missing"):
        assert _build.build(force=True) == _build.LIB
    assert made == ["library"] and pd.paged_decode_version() > 0
    with pytest.raises(RuntimeError, match="needs .*Python.h"):
        pd._step("attn_sinks")
    monkeypatch.setattr(_build.shutil, "which", lambda name: None)
    assert "compiler" in _build.bind_missing()
