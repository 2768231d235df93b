"""When the library and its extension module count as stale, on files with set times; nothing is compiled."""
import os

import pytest

import paged_gqa_decode_hpc_gb300 as hpc
from paged_gqa_decode_hpc_gb300 import _build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of its own: {name: path}; everything is current."""
    names = dict(LIB_PATH="lib.so", BINDING_PATH="binding.so", BINDING_SRC="csrc/binding.cpp", kernel="csrc/a.cu",
                 inner="csrc/a.h", header="include/hpc_decode.h", __file__="_build.py")
    paths = {k: tmp_path / v for k, v in names.items()}
    for p in paths.values():
        p.parent.mkdir(exist_ok=True)
        p.write_bytes(b"not a shared library")
    for k in ("LIB_PATH", "BINDING_PATH", "BINDING_SRC", "__file__"):
        monkeypatch.setattr(_build, k, str(paths[k]))
    monkeypatch.setattr(_build, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(_build, "INCLUDE", str(tmp_path / "include"))
    monkeypatch.setattr(_build, "_python_include", lambda: "/usr/include")
    at(paths, 100, "LIB_PATH", "BINDING_PATH")
    at(paths, 50, "BINDING_SRC", "kernel", "inner", "header", "__file__")
    return paths


def at(paths, t, *names):
    for n in names:
        os.utime(paths[n], (t, t))


def test_current(tree):
    assert not _build.is_stale()


@pytest.mark.parametrize("name", ["BINDING_SRC", "kernel", "inner", "header", "__file__"])
def test_a_changed_source(tree, name):
    at(tree, 150, name)
    assert _build.is_stale()


@pytest.mark.parametrize("name", ["BINDING_SRC", "header"])
def test_a_library_rebuilt_without_this_interpreters_module(tree, name):
    """Another interpreter, or one without headers, has rebuilt the library after the interface changed."""
    at(tree, 150, name)
    at(tree, 200, "LIB_PATH")
    assert _build.is_stale()


def test_no_module_and_no_headers_is_current(tree, monkeypatch):
    tree["BINDING_PATH"].unlink()
    assert _build.is_stale()
    monkeypatch.setattr(_build, "_python_include", lambda: None)
    assert not _build.is_stale()


@pytest.mark.parametrize("name", ["BINDING_SRC", "header"])
def test_an_old_module_is_not_loaded(tree, name, monkeypatch):
    monkeypatch.setattr(hpc, "_native", None)
    at(tree, 150, name)
    hpc._load_native(None)  # (loading the file would raise)
    assert hpc._native is None
