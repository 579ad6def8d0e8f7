"""The build script: what it leaves when a part of it fails.  The compilers are
stand-ins."""
import os
import stat
import sysconfig
import types

import pytest

import linear_recurrence_chunked_gated_amd as gdn
from linear_recurrence_chunked_gated_amd import _lib, build


def _script(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build into tmp_path whose hipcc writes an empty file at -o."""
    hipcc = _script(tmp_path / "hipcc", 'while [ "$1" != "-o" ]; do shift; done; : > "$2"\n')
    monkeypatch.setattr(build, "HIPCC", hipcc)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "calls.so"))
    return tmp_path


def test_library_is_linked_though_the_python_calls_fail(tree, monkeypatch):
    """The C library needs hipcc alone; a failure to build the module on
    torch's headers is raised after it is there."""
    monkeypatch.setenv("CXX", _script(tree / "cxx", "exit 1\n"))
    with pytest.raises(RuntimeError, match="sf_gdn_calls.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)


def test_a_failed_kernel_leaves_the_old_library(tree, monkeypatch):
    monkeypatch.setenv("CXX", _script(tree / "cxx", "exit 1\n"))
    monkeypatch.setattr(build, "HIPCC", _script(tree / "hipcc1", "exit 1\n"))
    (tree / "lib.so").write_text("old")
    with pytest.raises(RuntimeError, match="compile failed"):
        build.build()
    assert (tree / "lib.so").read_text() == "old"


def test_module_is_named_for_its_interpreter():
    assert os.path.basename(build.CALLS) == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    _lib.load_calls()
    assert gdn._calls.__file__ == build.CALLS


@pytest.mark.parametrize("stamp", [None, "0123456789abcdef"])
def test_module_of_another_header_is_refused(monkeypatch, stamp):
    """A module left from another build would pass structs that the library
    reads differently: it is refused before it is bound."""
    _lib.load_calls()
    bound = []
    old = types.SimpleNamespace(bind=lambda *a: bound.append(a), __file__="old")
    if stamp:
        old.INTERFACE = stamp
    monkeypatch.setattr(_lib, "_calls", None)
    monkeypatch.setattr(gdn, "_calls", old)
    with pytest.raises(RuntimeError, match="rebuild"):
        _lib.load_calls()
    assert not bound and _lib._calls is None


def test_a_missing_module_names_the_build(monkeypatch):
    """sys.modules holding None makes the import fail as a missing file does."""
    import sys
    _lib.load_calls()
    monkeypatch.setattr(_lib, "_calls", None)
    monkeypatch.delattr(gdn, "_calls")
    monkeypatch.setitem(sys.modules, gdn.__name__ + "._calls", None)
    with pytest.raises(RuntimeError, match="not built"):
        _lib.load_calls()
