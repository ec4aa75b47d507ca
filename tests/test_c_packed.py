"""The checkpoint and 4-bit calls from C: tests/c/packed_from_c.c is compiled
with gcc -std=c99 -pedantic against include/mhc.h, linked against the built
libmhc.so and run.  Every call returns before any device work, so no GPU is
needed."""
import os
import shutil
import subprocess

import pytest

from birkhoff_projection_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_c_caller(tmp_path):
    so = _lib.LIB_PATH
    assert os.path.exists(so), "build the library first (__graft_entry__.build())"
    exe = tmp_path / "packed_from_c"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror",
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c", "packed_from_c.c"),
                    "-o", str(exe), so, "-Wl,-rpath," + os.path.dirname(so)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "c packed ok" in r.stdout


def test_every_new_call_is_made():
    """Every function of the checkpoint and 4-bit sections of the header."""
    import re
    with open(os.path.join(ROOT, "include", "mhc.h"), encoding="utf-8") as f:
        text = f.read()
    section = text[text.index("* Activation checkpoints in 8 bits."):text.index("const char* mhc_status_string")]
    names = set(re.findall(r"^(?:mhc_status|int64_t) (mhc_\w+)\(", section, re.M))
    assert len(names) >= 17
    with open(os.path.join(ROOT, "tests", "c", "packed_from_c.c"), encoding="utf-8") as f:
        caller = f.read()
    assert not {n for n in names if n + "(" not in caller}
