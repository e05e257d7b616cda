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
