"""The build script: what it leaves when a part of it fails.  The compilers are
stand-ins."""
import os
import stat

import pytest

from linear_recurrence_chunked_gated_amd import build


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
