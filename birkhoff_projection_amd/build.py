"""Build the gfx950 shared library ``libmhc.so`` in-tree with hipcc, and the
extension module ``_binding.so`` that marshals PyTorch tensors to it.

Every HIP source is compiled for gfx950 only, with packed-fp32 code
generation switched off (``-target-feature -packed-fp32-ops``), then linked
into one shared library next to this file.  Run ``python -m
birkhoff_projection_amd.build`` or call :func:`build`.

The C library needs hipcc only: without PyTorch, run this file itself
(``python birkhoff_projection_amd/build.py``), which then leaves the extension
module out.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmhc.so")
SOURCES = ["abi.hip", "birkhoff.hip", "birkhoffn.hip", "mix.hip", "layer.hip", "ckpt.hip",
           "layer_ckpt.hip", "read.hip", "mx4.hip"]
BINDING = os.path.join(PKG, "_binding.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the gfx950 library cannot be built")


def compile_flags():
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC,
            "-Wall", "-Wno-unused-function"]


def binding_command(obj: str):
    """Compile command of csrc/binding.cpp (host code only, against torch)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], "/opt/rocm/include"]
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        raise RuntimeError("no C++ compiler: the tensor binding cannot be built")
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + \
        [f"-isystem{p}" for p in inc] + ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]


def binding_link(obj: str, out: str):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++" if shutil.which("g++") else "clang++", "-shared", "-o", out, obj, LIB, f"-L{lib}",
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"]


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _finish(procs, verbose):
    """Waits for the compilers; the names of the sources that failed."""
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or p.returncode != 0):
            print(out, end="", file=sys.stderr)
        if p.returncode != 0:
            failed.append(src)
    return failed


def _link(cmd, tmp, out, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)


def build(verbose: bool = False) -> str:
    """Compile every source and link ``libmhc.so``, then ``_binding.so`` where
    PyTorch is installed; returns the library's path.  The library is linked
    whatever becomes of the extension module, whose failure raises afterwards."""
    cc = hipcc()
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".hip", ".o"))
        objs.append(obj)
        procs.append((src, _start([cc] + compile_flags() + ["-c", os.path.join(CSRC, src), "-o", obj],
                                  verbose)))
    bobj = os.path.join(BUILD, "binding.o")
    binding, error = [], None
    if importlib.util.find_spec("torch") is None:
        print("no PyTorch: the library alone is built", file=sys.stderr)
    else:
        try:
            binding = [("binding.cpp", _start(binding_command(bobj), verbose))]
        except Exception as e:  # raised again once the library is linked
            error = e
    failed, bfailed = _finish(procs, verbose), _finish(binding, verbose)
    if failed:
        raise RuntimeError(f"compilation failed for {failed + bfailed}")
    tmp = LIB + ".tmp"
    _link([cc, f"--offload-arch={ARCH}", "-shared", "-Wl,-soname,libmhc.so", "-o", tmp] + objs, tmp, LIB,
          verbose)
    if error is not None:
        raise error
    if bfailed:
        raise RuntimeError(f"compilation failed for {bfailed}")
    if binding:
        tmp = BINDING + ".tmp"
        _link(binding_link(bobj, tmp), tmp, BINDING, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
