"""Argument errors of the 4-bit products and of the layer's read half, found
on the host before anything is enqueued (addresses are never dereferenced).
No GPU needed."""
import ctypes

import pytest

from birkhoff_projection_amd import _lib
from birkhoff_projection_amd._lib import LayerArgs

INVALID, UNSUPPORTED = 1, 2
A = [0x10000 + (k << 36) for k in range(12)]


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def _err(L):
    return L.mhc_last_error().decode()


def test_matmul_errors(L):
    def mm(ac=A[0], asc=A[1], bc=A[2], bs=A[3], o=A[4], dt=0, M=8, N=16, K=64):
        return L.mhc_mx4_matmul(ac, asc, bc, bs, o, dt, M, N, K, None)

    assert mm(None, None, None, None, None, M=0) == 0
    for kw, text in ((dict(K=48), "K must"), (dict(K=0), "K must"), (dict(N=12), "N must"), (dict(N=0), "N must"),
                     (dict(M=-1), "out of range"), (dict(M=1 << 28, N=1 << 20), "out of range"),
                     (dict(dt=2), "dtype"), (dict(ac=None), "NULL"), (dict(bs=A[3] + 4), "aligned"),
                     (dict(o=A[0] + 128), "overlaps"), (dict(o=A[3]), "overlaps")):
        assert mm(**kw) == INVALID, kw
        assert text in _err(L), (kw, _err(L))


def test_matmul_values_errors(L):
    W = L.mhc_mx4_matmul_values_workspace_bytes
    assert W(1, 16, 64) == 0 and W(512, 16, 64) > 0
    assert W(4, 12, 64) == -1 and W(4, 16, 40) == -1 and W(-1, 16, 64) == -1

    def mm(a=A[0], ad=0, bc=A[2], bs=A[3], o=A[4], dt=0, M=512, N=16, K=64, ws=A[5], n=1 << 20):
        return L.mhc_mx4_matmul_values(a, ad, bc, bs, o, dt, M, N, K, ws, n, None)

    for kw, text in ((dict(ad=4), "dtype"), (dict(dt=-1), "dtype"), (dict(K=33), "K must"), (dict(ws=None), "NULL"),
                     (dict(n=W(512, 16, 64) - 1), "workspace_bytes"), (dict(ws=A[0] + 64), "overlaps"),
                     (dict(ws=A[4]), "overlaps"), (dict(o=A[0]), "overlaps"), (dict(ws=A[5] + 8), "aligned")):
        assert mm(**kw) == INVALID, kw
        assert text in _err(L), (kw, _err(L))


def test_write_back_errors(L):
    def wb(p=A, T=8, n=4, C=64, K=64, xo=A[7], f=None):
        return L.mhc_mx4_write_back(p[0], p[1], p[2], p[3], p[4], p[5], p[6], xo, f, T, n, C, K, None)

    assert wb([None] * 8, T=0, xo=None) == 0
    assert wb(n=3) == UNSUPPORTED
    for kw, text in ((dict(C=60), "C must"), (dict(K=16), "K must"), (dict(T=-1), "out of range"),
                     (dict(xo=None), "NULL"), (dict(xo=A[4]), "overlaps"), (dict(f=A[7] + 64), "overlaps"),
                     (dict(f=A[8] + 2), "aligned")):
        assert wb(**kw) == INVALID, kw
        assert text in _err(L), (kw, _err(L))


def test_layer_read_errors(L):
    W = L.mhc_layer_read_workspace_bytes
    assert W(1, 4, 64) > 0 and W(2048, 4, 64) > 0 and W(2049, 4, 64) == 0 and W(16, 3, 64) == -1

    def args(T=16, C=64):
        a = LayerArgs()
        a.T, a.n, a.C, a.eps = T, 4, C, 1e-6
        for i, name in enumerate(("x", "W", "u", "rms", "logits", "H_pre", "H_post", "H_res", "workspace")):
            setattr(a, name, 0x10000 + (i << 32))
        a.workspace_bytes = 1 << 20
        return a

    assert L.mhc_layer_read(None, None, None, None) == INVALID
    assert L.mhc_layer_read(ctypes.byref(args(T=0)), None, None, None) == 0
    for field, value in (("C", 96), ("T", -1), ("eps", 0.0), ("x", None), ("u", None), ("rms", 0x10002),
                         ("logits", 0x10000), ("workspace", None), ("workspace_bytes", W(16, 4, 64) - 1)):
        a = args()
        setattr(a, field, value)
        assert L.mhc_layer_read(ctypes.byref(a), None, None, None) == INVALID, field
    a = args()
    a.n = 2
    assert L.mhc_layer_read(ctypes.byref(a), None, None, None) == UNSUPPORTED
    assert L.mhc_layer_read(ctypes.byref(args()), A[9], None, None) == INVALID and "together" in _err(L)
    assert L.mhc_layer_read(ctypes.byref(args()), A[9], 0x10000, None) == INVALID and "overlaps" in _err(L)


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import birkhoff_projection_amd as bp
    q = lambda r, c: (torch.zeros(r, c // 2, dtype=torch.uint8), torch.zeros(r, c // 32, dtype=torch.uint8))
    with pytest.raises(TypeError):
        bp.mx4_matmul(q(4, 64), q(8, 64))  # host tensors
    with pytest.raises(ValueError):
        bp.mx4_linear(torch.zeros(31, 64), torch.zeros(32, 64))
    with pytest.raises(ValueError):
        bp.mx4_linear(torch.zeros(2, 32, 64), torch.zeros(32, 64))
    with pytest.raises(TypeError):
        bp.layer_read(torch.zeros(4, 4, 64), torch.zeros(24, 256))


def test_joint_quantisation_errors(L):
    def both(p=A, dt=0, R=64, C=64):
        return L.mhc_mx4_quantize_both(p[0], dt, p[1], p[2], p[3], p[4], R, C, None)

    def ckpt(p=A, dt=0, R=64, C=64, fmt=0):
        return L.mhc_mx4_quantize_ckpt(p[0], dt, p[1], p[2], p[3], p[4], R, C, fmt, None)

    def again(p=A, R=64, C=64, fmt=0):
        return L.mhc_mx4_requantize(p[0], p[1], p[2], p[3], R, C, fmt, None)

    none = [None] * 5
    assert both(none, R=0) == 0 and ckpt(none, R=0) == 0 and again(none, R=0) == 0

    def at(k, v):
        return A[:k] + [v] + A[k + 1:]

    for f, kw, text in ((both, dict(R=40), "R must"), (both, dict(C=40), "C must"), (both, dict(dt=3), "dtype"),
                        (both, dict(R=-32), "out of range"), (both, dict(p=at(3, None)), "NULL"),
                        (both, dict(p=at(4, A[2])), "overlaps"), (both, dict(p=at(3, A[0] + 16)), "overlaps"),
                        (ckpt, dict(C=40), "C must"), (ckpt, dict(fmt=2), "format"), (ckpt, dict(dt=-1), "dtype"),
                        (ckpt, dict(p=at(1, A[3])), "overlaps"), (ckpt, dict(p=at(4, A[4] + 2)), "aligned"),
                        (again, dict(R=48), "R must"), (again, dict(C=0), "C must"), (again, dict(fmt=-1), "format"),
                        (again, dict(C=128 * 65536, R=32), "out of range"), (again, dict(p=at(2, A[0])), "overlaps"),
                        (again, dict(p=at(1, None)), "NULL")):
        assert f(**kw) == INVALID, (f.__name__, kw)
        assert text in _err(L), (f.__name__, kw, _err(L))
