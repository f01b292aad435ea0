"""The build's own rules, with compilers that only touch their output."""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import subprocess
import sysconfig
import types

import pytest

import prompt_lookup_speculative_gb300 as pkg
from prompt_lookup_speculative_gb300 import build as lib_build


@pytest.fixture
def build_dir(tmp_path, monkeypatch):
    """The build in a folder of its own, each compiler a command that makes its file."""
    for name in ("LIB_PATH", "CHECKED_LIB_PATH"):
        monkeypatch.setattr(lib_build, name, str(tmp_path / os.path.basename(getattr(lib_build, name))))
    monkeypatch.setattr(lib_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(lib_build, "compile_command", lambda out, extra=None, checked=False: ["touch", out])
    monkeypatch.setattr(lib_build, "binding_command", lambda out: ["touch", out])
    return tmp_path


def fake_torch(tmp_path, monkeypatch, cuda: bool):
    """An installed PyTorch, built with CUDA or without."""
    root = tmp_path / "site" / "torch"
    (root / "lib").mkdir(parents=True)
    (root / "lib" / "libc10.so").touch()
    if cuda:
        (root / "lib" / "libc10_cuda.so").touch()
    find = importlib.util.find_spec
    spec = types.SimpleNamespace(origin=str(root / "__init__.py"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9")


def test_a_pytorch_without_cuda_gets_no_entry(build_dir, monkeypatch):
    """Its libraries cannot be linked against: the C libraries are built all the same, and
    a call says what is missing."""
    fake_torch(build_dir, monkeypatch, cuda=False)
    monkeypatch.setattr(lib_build, "binding_command", lambda out: ["false"])
    assert lib_build.binding_path() is None
    assert lib_build.build() == lib_build.LIB_PATH
    assert os.path.exists(lib_build.LIB_PATH) and os.path.exists(lib_build.CHECKED_LIB_PATH)
    assert lib_build.up_to_date()
    monkeypatch.setattr(pkg, "load_library", lambda: None)
    monkeypatch.setattr(pkg, "_target_module", None)
    with pytest.raises(RuntimeError, match="CUDA"):
        pkg._target()


def test_an_entry_that_does_not_compile_leaves_the_libraries(build_dir, monkeypatch):
    """The error is raised, the libraries are in place, and no entry of an older build
    stays beside them."""
    fake_torch(build_dir, monkeypatch, cuda=True)
    open(lib_build.binding_path(), "w").close()
    monkeypatch.setattr(lib_build, "binding_command", lambda out: ["false"])
    with pytest.raises(subprocess.CalledProcessError):
        lib_build.build(force=True)
    assert os.path.exists(lib_build.LIB_PATH) and os.path.exists(lib_build.CHECKED_LIB_PATH)
    assert not os.path.exists(lib_build.binding_path()) and not lib_build.up_to_date()


def test_a_library_that_does_not_compile_replaces_nothing(build_dir, monkeypatch):
    fake_torch(build_dir, monkeypatch, cuda=True)
    monkeypatch.setattr(lib_build, "compile_command", lambda out, extra=None, checked=False: ["false"])
    with pytest.raises(subprocess.CalledProcessError):
        lib_build.build(force=True)
    assert not os.path.exists(lib_build.LIB_PATH) and not os.path.exists(lib_build.binding_path())


def test_the_entrys_name_tells_the_python_and_the_pytorch(build_dir, monkeypatch):
    """Another Python in the same tree must not load what was built for this one."""
    fake_torch(build_dir, monkeypatch, cuda=True)
    mine = lib_build.binding_path()
    var = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: {"EXT_SUFFIX": ".cpython-399-x.so"}.get(name, var(name)))
    assert lib_build.binding_path() != mine and "9.9" in os.path.basename(mine)
    lib_build.build(force=True)
    monkeypatch.undo()
    assert sysconfig.get_config_var("EXT_SUFFIX") in mine
