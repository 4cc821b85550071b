"""The build without a working torch or C++ compiler: the libraries need hipcc alone (stand-in compilers, no GPU)."""

from __future__ import annotations

import os
import sys

import pytest

from persistent_gemm_amd import build as b


def _compiler(path, body):
    path.write_text("#!/bin/sh\n" + body)
    path.chmod(0o755)
    return str(path)


# writes its name into the file after -o
WRITES = 'while [ "$1" != -o ]; do shift; done\necho built > "$2"\n'


@pytest.fixture
def tree(tmp_path, monkeypatch):
    (tmp_path / "csrc").mkdir()
    monkeypatch.setattr(b, "CSRC", str(tmp_path / "csrc"))
    for name in ("LIB", "PROBE_LIB", "NATIVE"):
        monkeypatch.setattr(b, name, str(tmp_path / name))
    monkeypatch.setattr(b, "HIPCC", _compiler(tmp_path / "hipcc", WRITES))
    monkeypatch.setattr(b, "CXX", _compiler(tmp_path / "cxx", WRITES))
    return tmp_path


def test_everything(tree):
    assert b.build() == str(tree / "LIB")
    assert all((tree / n).exists() for n in ("LIB", "PROBE_LIB", "NATIVE"))


@pytest.mark.parametrize("why", ["the compiler fails", "no compiler", "no torch"])
def test_libraries_without_the_native_binding(tree, monkeypatch, capfd, why):
    if why == "the compiler fails":
        monkeypatch.setattr(b, "CXX", _compiler(tree / "cxx", "echo no header; exit 1\n"))
    elif why == "no compiler":
        monkeypatch.setattr(b, "CXX", str(tree / "absent"))
    else:
        monkeypatch.setitem(sys.modules, "torch", None)
    (tree / "NATIVE").write_text("of another version")
    assert b.build() == str(tree / "LIB")
    assert (tree / "LIB").exists() and (tree / "PROBE_LIB").exists()
    assert not (tree / "NATIVE").exists()       # none rather than an old one
    assert "native binding" in capfd.readouterr().err


def test_a_library_that_does_not_compile(tree, monkeypatch):
    monkeypatch.setattr(b, "HIPCC", _compiler(tree / "hipcc", "exit 1\n"))
    with pytest.raises(RuntimeError, match="build failed"):
        b.build()
    assert not os.path.exists(b.LIB)


def test_calls_without_the_native_binding_say_so(monkeypatch):
    import persistent_gemm_amd as pg
    monkeypatch.setattr(pg, "_NATIVE", None)
    monkeypatch.delattr(pg, "_sknative", raising=False)
    monkeypatch.setitem(sys.modules, "persistent_gemm_amd._sknative", None)
    with pytest.raises(RuntimeError, match="native binding"):
        pg.quantize_fp8_block(None)
    assert pg.plan(pg.MXFP4, 256, 256, 512, num_cus=256).grid > 0      # and the others go on
