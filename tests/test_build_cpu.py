"""Building: the C library needs neither a host compiler of its own nor PyTorch's headers, and the native half of
the binding belongs to the interpreter and the PyTorch that it was compiled against."""

from __future__ import annotations

import sys

import pytest

from paged_kv_cache_244_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def test_the_c_library_builds_without_a_host_compiler(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "NATIVE", tmp_path / "_pa_torch.so")
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    with pytest.warns(RuntimeWarning, match="no-such-compiler"):
        assert _build.build() == _build.LIBRARY
    assert not _build.NATIVE.exists()


def test_the_c_library_builds_without_pytorch(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "NATIVE", tmp_path / "_pa_torch.so")
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr(_build, "torch_dir", lambda: None, raising=False)
    with pytest.warns(RuntimeWarning, match="PyTorch"):
        assert _build.build() == _build.LIBRARY
    assert not _build.NATIVE.exists()


def test_the_native_half_belongs_to_its_pytorch_and_interpreter(monkeypatch, tmp_path):
    assert _build.native_up_to_date()
    other = tmp_path / "torch"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '9.9.9'\n")
    with monkeypatch.context() as m:
        m.setattr(_build, "torch_dir", lambda: other)
        assert not _build.native_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-399-other")
        assert not _build.native_up_to_date()
    assert _build.native_up_to_date()


def test_a_native_half_that_does_not_load_says_why(monkeypatch):
    from paged_kv_cache_244_gb300 import binding
    import paged_kv_cache_244_gb300 as package
    monkeypatch.setattr(binding, "_native_module", None)
    monkeypatch.setitem(sys.modules, "paged_kv_cache_244_gb300._pa_torch", None)
    monkeypatch.delattr(package, "_pa_torch", raising=False)
    with pytest.raises(RuntimeError, match="_pa_torch.so cannot be loaded .*import of"):
        binding._native()
