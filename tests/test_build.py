"""Building the library and the torch binding, with small sources in their place."""

import ctypes
import importlib.metadata
import os
import sys

import pytest

from software_pipelined_tiled_02_gb300 import build as tbuild


@pytest.fixture
def small(tmp_path, monkeypatch):
    source = tmp_path / "one.cu"
    source.write_text('extern "C" int one() { return 1; }\n')
    binding = tmp_path / "binding.cpp"
    binding.write_text('extern "C" int two() { return 2; }\n')
    for name, value in (("LIB", "libone.so"), ("LIB_DEBUG", "libone_debug.so"), ("BINDING", "_two.so"),
                        ("BINDING_MADE_FOR", "_two.made_for")):
        monkeypatch.setattr(tbuild, name, str(tmp_path / value), raising=False)
    monkeypatch.setattr(tbuild, "SOURCES", [str(source)])
    monkeypatch.setattr(tbuild, "DEPS", [str(source)])
    monkeypatch.setattr(tbuild, "BINDING_SOURCE", str(binding))
    return binding


def test_the_library_needs_no_torch(small, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    lib = tbuild.build()
    assert ctypes.CDLL(lib).one() == 1
    assert not os.path.exists(tbuild.BINDING)
    assert "torch" in capsys.readouterr().err


def test_a_binding_that_fails_leaves_the_library_and_no_process(small):
    psutil = pytest.importorskip("psutil")
    small.write_text("this is no C++\n")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        tbuild.build()
    assert ctypes.CDLL(tbuild.LIB).one() == 1 and not os.path.exists(tbuild.BINDING)
    assert not [p for p in psutil.Process().children() if p.name() in ("nvcc", "g++")]


def test_a_compiler_that_does_not_start_leaves_the_library(small, monkeypatch):
    monkeypatch.setattr(tbuild, "binding_command", lambda out: ["/no/such/compiler", out])
    with pytest.raises(RuntimeError, match="does not start"):
        tbuild.build()
    assert ctypes.CDLL(tbuild.LIB).one() == 1


def test_another_torch_makes_the_binding_stale(small, monkeypatch):
    tbuild.build()
    assert tbuild.up_to_date(tbuild.LIB) and tbuild.up_to_date(tbuild.BINDING)
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.1+other")
    assert tbuild.up_to_date(tbuild.LIB) and not tbuild.up_to_date(tbuild.BINDING)
    tbuild.build()
    assert tbuild.up_to_date(tbuild.BINDING)
