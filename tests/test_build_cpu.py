"""What the build needs, and what it leaves where a part of it fails."""
import importlib.util
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """A copy of the build script of its own that puts one small source's library into
    tmp_path."""
    spec = importlib.util.spec_from_file_location(
        "_build_copy", os.path.join(ROOT, "sp_boundary_norm_gb300", "_build.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    source = tmp_path / "one.cu"
    source.write_text('extern "C" int one() { return 1; }\n')
    out = tmp_path / "out"
    monkeypatch.setattr(module, "OUT_DIR", str(out))
    monkeypatch.setattr(module, "LIB_PATH", str(out / "lib.so"))
    monkeypatch.setattr(module, "MODULE_PATH", str(out / "mod.so"))
    monkeypatch.setattr(module, "_sources", lambda: [str(source)])
    return module


def without_torch(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)


def test_the_library_needs_no_torch(build, monkeypatch):
    without_torch(monkeypatch)
    spec = importlib.util.spec_from_file_location("_build_again", build.__file__)
    spec.loader.exec_module(importlib.util.module_from_spec(spec))     # imports none
    assert os.path.exists(build.build_library())
    assert build.build_module() is None and not os.path.exists(build.MODULE_PATH)


def test_a_failing_host_compiler_leaves_the_library(build, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="host compiler"):
        build.build_library()
    made = os.stat(build.LIB_PATH).st_mtime_ns
    with pytest.raises(RuntimeError, match="host compiler"):
        build.build_library()
    assert os.stat(build.LIB_PATH).st_mtime_ns == made      # and it is not built again


def test_the_module_is_the_interpreters_own(build, monkeypatch, tmp_path):
    """Another Python or torch version builds the module again, and the module alone."""
    compiler = tmp_path / "cxx"
    compiler.write_text('#!/bin/sh\necho run >> "%s"\nwhile [ "$1" != -o ]; do shift; done\n'
                        ': > "$2"\n' % (tmp_path / "runs"))
    compiler.chmod(0o755)
    monkeypatch.setenv("CXX", str(compiler))
    runs = lambda: (tmp_path / "runs").read_text().count("run")
    build.build_library()
    made = os.stat(build.LIB_PATH).st_mtime_ns
    build.build_library()
    assert runs() == 1
    monkeypatch.setattr(build.sys, "version", "another")
    build.build_library()
    build.build_library()
    assert runs() == 2 and os.stat(build.LIB_PATH).st_mtime_ns == made
