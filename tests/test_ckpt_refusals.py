"""Argument errors of the checkpoint and 4-bit quantisation calls, found on
the host before anything is enqueued (addresses are never dereferenced).  No
GPU needed."""
import ctypes

import pytest

from birkhoff_projection_amd import _lib
from birkhoff_projection_amd._lib import LayerArgs, LayerCkpt, ProjOpts

INVALID, UNSUPPORTED = 1, 2
A = [0x10000 + (k << 34) for k in range(20)]  # far apart, aligned


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def _err(L):
    return L.mhc_last_error().decode()


def test_empty_batches(L):
    assert L.mhc_ckpt_pack(None, 0, None, None, 0, 8, 0, None) == 0
    assert L.mhc_ckpt_unpack(None, None, None, 1, 0, 8, 1, None) == 0
    assert L.mhc_stream_mix_ckpt(None, None, None, None, None, None, 0, 4, 8, 0, None, None) == 0
    assert L.mhc_stream_mix_bwd_ckpt(None, None, None, None, None, None, 0, 4, 8, 0, None) == 0
    assert L.mhc_mx4_quantize(None, 0, None, None, 0, 32, 0, None) == 0
    assert L.mhc_mx4_dequantize(None, None, None, 0, 0, 32, None) == 0


def test_pack_errors(L):
    def pack(x=A[0], dt=0, c=A[1], s=A[2], R=5, C=64, fmt=0):
        return L.mhc_ckpt_pack(x, dt, c, s, R, C, fmt, None)

    def unpack(c=A[1], s=A[2], x=A[0], dt=0, R=5, C=64, fmt=0):
        return L.mhc_ckpt_unpack(c, s, x, dt, R, C, fmt, None)

    for f in (pack, unpack):
        for kw, text in ((dict(dt=2), "dtype"), (dict(fmt=2), "format"), (dict(fmt=-1), "format"),
                         (dict(C=60), "multiple of 8"), (dict(C=0), "multiple of 8"),
                         (dict(R=-1), "out of range"), (dict(R=1 << 40), "out of range"),
                         (dict(R=(1 << 33) // 8 + 1), "out of range"),
                         (dict(x=None), "NULL"), (dict(s=None), "NULL"), (dict(c=A[1] + 8), "aligned"),
                         (dict(c=A[0] + 16), "overlaps"), (dict(s=A[1] + 64), "overlaps")):
            assert f(**kw) == INVALID, kw
            assert text in _err(L), (kw, _err(L))


def test_mix_errors(L):
    def fwd(n=4, T=5, C=64, fmt=0, H_out=None, out=A[2], codes=A[3], opts=None, x=A[0]):
        return L.mhc_stream_mix_ckpt(x, A[1], H_out, out, codes, A[4], T, n, C, fmt, opts, None)

    assert fwd(n=3) == UNSUPPORTED
    for kw in (dict(T=-1), dict(C=60), dict(C=4), dict(fmt=2), dict(out=A[0] + 256), dict(out=None),
               dict(codes=A[2]), dict(codes=A[1] + 32), dict(x=A[0] + 2)):
        assert fwd(**kw) == INVALID, kw
    o = ProjOpts()
    L.mhc_proj_opts_default(ctypes.byref(o))
    assert fwd(H_out=A[2] + 32, opts=ctypes.byref(o)) == INVALID and "overlaps" in _err(L)
    assert fwd(H_out=A[1] + 64, opts=ctypes.byref(o)) == INVALID
    o.tol = -1.0
    assert fwd(opts=ctypes.byref(o)) == INVALID and "tol" in _err(L)

    def bwd(n=4, T=5, C=64, fmt=0, codes=A[0], gx=A[4], gH=A[5]):
        return L.mhc_stream_mix_bwd_ckpt(codes, A[1], A[2], A[3], gx, gH, T, n, C, fmt, None)

    assert bwd(n=5) == UNSUPPORTED
    for kw in (dict(T=-1), dict(C=60), dict(fmt=7), dict(codes=None), dict(gx=A[3]), dict(gx=A[0] + 16),
               dict(gH=A[2]), dict(gH=A[5] + 4)):
        assert bwd(**kw) == INVALID, kw


def _layer(T=16, C=64):
    a, k = LayerArgs(), LayerCkpt()
    a.T, a.n, a.C, a.eps = T, 4, C, 1e-6
    names = [n for n, _ in LayerArgs._fields_[5:-1]]
    for i, n in enumerate(names):
        setattr(a, n, A[0] + (i << 32))
    for i, n in enumerate(("x_codes", "x_scales", "f_codes", "f_scales")):
        setattr(k, n, A[0] + ((40 + i) << 32))
    a.workspace_bytes = 1 << 30
    return a, k


def test_layer_errors(L):
    assert L.mhc_layer_ckpt_workspace_bytes(16, 3, 64) == -1
    assert L.mhc_layer_ckpt_workspace_bytes(16, 4, 60) == -1
    assert L.mhc_layer_ckpt_workspace_bytes(16, 4, 64) > 0
    for f in (L.mhc_layer_fwd_ckpt, L.mhc_layer_bwd_ckpt):
        a, k = _layer()
        assert f(None, ctypes.byref(k), None) == INVALID
        assert f(ctypes.byref(a), None, None) == INVALID
        for obj, field, value in ((a, "C", 96), (a, "T", -1), (k, "format", 2), (k, "x_codes", None),
                                  (k, "f_scales", A[0] + (43 << 32) + 8), (a, "logits", k.x_codes),
                                  (k, "f_codes", k.x_codes)):
            a, k = _layer()
            setattr(a if isinstance(obj, LayerArgs) else k, field, value)
            assert f(ctypes.byref(a), ctypes.byref(k), None) == INVALID, field
        a, k = _layer()
        a.n = 3
        assert f(ctypes.byref(a), ctypes.byref(k), None) == UNSUPPORTED
        a, k = _layer(T=0)
        assert f(ctypes.byref(a), ctypes.byref(k), None) == 0
    assert L.mhc_layer_read_workspace_bytes(0, 4, 64) == 0  # no tokens
    assert L.mhc_layer_read_workspace_bytes(2049, 4, 64) == 0
    assert L.mhc_layer_ckpt_workspace_bytes(0, 4, 64) >= 0
    a, k = _layer()
    a.workspace_bytes = L.mhc_layer_read_workspace_bytes(16, 4, 64) - 1
    assert L.mhc_layer_fwd_ckpt(ctypes.byref(a), ctypes.byref(k), None) == INVALID
    assert "workspace_bytes" in _err(L)
    a, k = _layer()
    a.eps = 0.0
    assert L.mhc_layer_fwd_ckpt(ctypes.byref(a), ctypes.byref(k), None) == INVALID
    a, k = _layer()
    a.workspace_bytes = L.mhc_layer_ckpt_workspace_bytes(16, 4, 64) - 1
    assert L.mhc_layer_bwd_ckpt(ctypes.byref(a), ctypes.byref(k), None) == INVALID
    assert "workspace_bytes" in _err(L)
    a, k = _layer()
    a.workspace = a.workspace + 16
    assert L.mhc_layer_bwd_ckpt(ctypes.byref(a), ctypes.byref(k), None) == INVALID


def test_mx4_quantize_errors(L):
    def q(x=A[0], dt=0, c=A[1], s=A[2], R=64, C=64, tr=0):
        return L.mhc_mx4_quantize(x, dt, c, s, R, C, tr, None)

    for kw, text in ((dict(dt=3), "dtype"), (dict(tr=2), "transpose"), (dict(C=40), "multiple of 32"),
                     (dict(C=44, tr=1), "multiple of 8"), (dict(R=40, tr=1), "R must be"),
                     (dict(C=64 * 65536, tr=1, R=32), "out of range"), (dict(R=-32), "out of range"),
                     (dict(c=A[0]), "overlaps"), (dict(x=None), "NULL"), (dict(s=A[2] + 4), "aligned")):
        assert q(**kw) == INVALID, kw
        assert text in _err(L), (kw, _err(L))
    assert L.mhc_mx4_dequantize(A[0], A[1], A[2], 0, 4, 40, None) == INVALID
    assert L.mhc_mx4_dequantize(A[0], A[1], A[0] + 16, 0, 4, 64, None) == INVALID
    assert L.mhc_mx4_dequantize(A[0], A[1], A[2], 5, 4, 64, None) == INVALID


def test_layer_ckpt_struct_layout_matches_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [f for f, _ in LayerCkpt._fields_]
    src = tmp_path / "off.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mhc.h"\nint main(void){\n'
                   + "".join(f'printf("%zu\\n", offsetof(mhc_layer_ckpt, {f}));\n' for f in fields)
                   + 'printf("%zu\\n", sizeof(mhc_layer_ckpt));\nreturn 0;}\n')
    exe = tmp_path / "off"
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(LayerCkpt, f).offset for f in fields] + [ctypes.sizeof(LayerCkpt)]


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    import birkhoff_projection_amd as bp
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bp.ckpt_pack(x)
    with pytest.raises(ValueError):
        bp.ckpt_pack(x, format="fp8")
    with pytest.raises(TypeError):
        bp.ckpt_pack(x.half())
    with pytest.raises(TypeError):
        bp.mx4_quantize(x)
    with pytest.raises(TypeError):
        bp.ckpt_unpack(torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(3, 2, dtype=torch.uint8),
                       dtype=torch.float16)
