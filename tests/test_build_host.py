"""When the build compiles the extension of the training operators, and when it leaves it out."""
import importlib.util
import os
import types

import pytest

from conftest import ROOT


@pytest.fixture
def B():
    path = os.path.join(ROOT, "routing_grouped_gemm_router_gb300", "build.py")
    spec = importlib.util.spec_from_file_location("_build_under_test", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_extension_is_left_out_without_pytorch_s_cuda_libraries(B, monkeypatch, tmp_path):
    (tmp_path / "lib").mkdir()
    spec = types.SimpleNamespace(origin=str(tmp_path / "__init__.py"))
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: spec)
    assert B._torch_dir() is None and B._native_up_to_date()
    (tmp_path / "lib" / "libc10_cuda.so").touch()
    assert B._torch_dir() == str(tmp_path)
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: None)
    assert B._torch_dir() is None


def test_an_extension_for_another_python_or_pytorch_is_built_again(B, monkeypatch, tmp_path):
    if B._torch_dir() is None:
        pytest.skip("no PyTorch with CUDA libraries")
    native, mark = tmp_path / "_native.so", tmp_path / "native_for.txt"
    native.touch()  # newer than every source
    monkeypatch.setattr(B, "NATIVE", str(native))
    monkeypatch.setattr(B, "NATIVE_FOR", str(mark), raising=False)
    assert not B._native_up_to_date()  # not known what it is for
    mark.write_text(B._native_for())
    assert B._native_up_to_date()
    monkeypatch.setattr(B.importlib.metadata, "version", lambda name: "2.0.0")
    assert not B._native_up_to_date()
    monkeypatch.undo()
    monkeypatch.setattr(B, "NATIVE", str(native))
    monkeypatch.setattr(B, "NATIVE_FOR", str(mark))
    monkeypatch.setattr(B.sys, "version", "3.9.0")
    assert not B._native_up_to_date()
