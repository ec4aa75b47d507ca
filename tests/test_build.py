"""The build's own steps, with stand-ins for the compilers: the C library
needs neither PyTorch nor a host compiler that fits it.  No GPU needed."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD_PY = os.path.join(ROOT, "birkhoff_projection_amd", "build.py")

FAKE_CC = """#!/bin/sh
# writes what -o names
while [ $# -gt 0 ]; do
  if [ "$1" = "-o" ]; then echo built > "$2"; fi
  shift
done
"""


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py loaded by its path (the package is not imported), with every
    output below tmp_path and a stand-in for hipcc."""
    cc = tmp_path / "hipcc"
    cc.write_text(FAKE_CC)
    cc.chmod(0o755)
    monkeypatch.setenv("HIPCC", str(cc))
    spec = importlib.util.spec_from_file_location("build_under_test", BUILD_PY)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for name, at in (("BUILD", "_build"), ("LIB", "libmhc.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(m, name, str(tmp_path / at))
    return m


def test_library_without_torch(build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # as if it were not installed
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_library_without_a_host_compiler(build, monkeypatch):
    def none(obj):
        raise RuntimeError("no C++ compiler")
    monkeypatch.setattr(build, "binding_command", none)
    with pytest.raises(RuntimeError, match="no C\\+\\+ compiler"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_library_where_the_module_does_not_compile(build, monkeypatch, capsys):
    monkeypatch.setattr(build, "binding_command", lambda obj: ["sh", "-c", "echo does not fit; exit 1"])
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "does not fit" in capsys.readouterr().err


def test_both(build, monkeypatch, tmp_path):
    pytest.importorskip("torch")
    cc = str(tmp_path / "hipcc")
    monkeypatch.setattr(build, "binding_command", lambda obj: [cc, "-o", obj])
    monkeypatch.setattr(build, "binding_link", lambda obj, out: [cc, "-o", out])
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)


def test_a_kernel_that_does_not_compile_fails(build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr(build, "hipcc", lambda: "false")
    with pytest.raises(RuntimeError, match="mx4.hip"):
        build.build()
    assert not os.path.exists(build.LIB)


def test_runs_as_a_file_without_the_package(tmp_path):
    """What a C user without PyTorch runs; only its compiler is a stand-in."""
    code = ("import runpy, sys, os; sys.modules['torch'] = None; "
            f"m = runpy.run_path({BUILD_PY!r}); print(len(m['SOURCES']), 'birkhoff_projection_amd' in sys.modules)")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=tmp_path)
    assert r.returncode == 0 and r.stdout.split()[1] == "False", r.stdout + r.stderr
