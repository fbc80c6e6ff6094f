"""What build() asks of a machine, with stand-ins for the compilers: the library
needs nvcc alone; the extension module belongs to one torch."""
import os
import stat

import pytest

from deterministic_w8a8_int8_gb300 import build as b


@pytest.fixture
def box(tmp_path, monkeypatch):
    """A machine whose nvcc and g++ write their output file and nothing else."""
    tools, pkg = tmp_path / "cuda" / "bin", tmp_path / "pkg"
    for d in (tools, pkg, tmp_path / "cuda" / "lib64"):
        d.mkdir(parents=True)
    for name in ("nvcc", "g++"):
        tool = tools / name
        tool.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && echo made > "$2"; shift; done\n')
        tool.chmod(tool.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(b, "_nvcc", lambda: str(tools / "nvcc"))
    monkeypatch.setenv("CXX", str(tools / "g++"))
    monkeypatch.setattr(b, "BUILD_DIR", str(pkg / "_build"))
    monkeypatch.setattr(b, "LIB_PATH", str(pkg / "libprism.so"))
    monkeypatch.setattr(b, "MODULE_PATH", str(pkg / "_decode.so"))
    monkeypatch.setattr(b, "STAMP_PATH", str(pkg / "_build" / "decode_py.stamp"), raising=False)
    return tmp_path


def _torch(monkeypatch, path, version):
    (path / "include" / "torch" / "csrc").mkdir(parents=True, exist_ok=True)
    (path / "version.py").write_text(f"__version__ = '{version}'\n")
    monkeypatch.setattr(b, "_torch_dir", lambda: str(path))


def test_the_library_without_torch(box, monkeypatch):
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    with pytest.warns(UserWarning, match="torch's headers"):
        assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.MODULE_PATH)
    assert b.up_to_date()


def test_the_library_without_a_cxx_compiler(box, monkeypatch):
    monkeypatch.delenv("CXX")
    monkeypatch.setattr(b.shutil, "which", lambda name: None)
    with pytest.warns(UserWarning, match="g\\+\\+"):
        assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.MODULE_PATH)


def test_another_torch_needs_another_module(box, monkeypatch):
    _torch(monkeypatch, box / "torch", "2.9.1")
    b.build()
    assert os.path.exists(b.MODULE_PATH) and b.up_to_date()
    _torch(monkeypatch, box / "torch", "2.11.0")
    assert not b.up_to_date()
    b.build()
    assert b.up_to_date()
