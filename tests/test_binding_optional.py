"""The package without its native binding (no g++ or headers, a file that does not load): everything
goes through ctypes."""
import os

import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from paged_mla_decode_07_gb300 import builder


@pytest.fixture
def unloaded(monkeypatch):
    mla.build()
    monkeypatch.setattr(mla, "_lib", None)
    monkeypatch.setattr(mla, "_native", None)


@pytest.mark.parametrize("content", [None, b"not a shared library"])
def test_the_library_loads_without_the_binding(monkeypatch, tmp_path, unloaded, content):
    path = tmp_path / "_mla_binding.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(builder, "BINDING", str(path))
    with pytest.warns(RuntimeWarning, match="through ctypes"):
        assert mla.lib().mla_abi_version() == 3
    assert mla._native is None
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        mla.window_decode(z, z, z, z, 1.0, window=1)


def test_a_binding_that_does_not_build_is_a_warning(monkeypatch, tmp_path):
    mla.build()
    monkeypatch.setattr(builder, "BINDING", str(tmp_path / "_mla_binding.so"))
    monkeypatch.setattr(builder, "build_library", lambda verbose: pytest.fail("the library is up to date"))
    monkeypatch.setenv("PATH", str(tmp_path))  # no g++
    with pytest.warns(RuntimeWarning, match="not built"):
        assert builder.build() == builder.LIB
    assert not os.path.exists(builder.BINDING)


def test_a_library_that_does_not_build_is_an_error(monkeypatch, tmp_path):
    monkeypatch.setattr(builder, "BUILD", str(tmp_path))
    monkeypatch.setattr(builder, "LIB", str(tmp_path / "libmla.so"))
    monkeypatch.setattr(builder, "BINDING", str(tmp_path / "_mla_binding.so"))
    monkeypatch.setattr(builder, "SOURCES", ["missing.cu"])
    monkeypatch.setattr(builder, "compile_binding", lambda: "binding.o")
    with pytest.raises(RuntimeError, match="missing.cu"):
        builder.build()
    assert not os.path.exists(builder.LIB)
