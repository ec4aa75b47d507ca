"""Python entry points over the checkpoint and 4-bit calls of the C ABI.

Like ``ops``: every function takes CUDA (HIP) tensors, checks dtype, shape,
contiguity and device, passes raw pointers and torch's current stream to
``libmhc.so`` and returns the output tensors.  A packed tensor is a pair
``(codes, scales)`` of uint8 tensors: one scale byte s, standing for
2^(s - 127), for each 32 consecutive values of a row.

8-bit checkpoints have ``format`` "e4m3" (8-bit floating point) or "int8"
(multiples of 1/64 of the scale) and codes of the values' shape.  4-bit
(MXFP4) codes hold two values a byte, the even one in the low half.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from ._lib import LayerArgs, LayerCkpt, check, lib
from .ops import (_bwd_shapes, _dict_out, _fwd_shapes, _layer_args, _need, _out, birkhoff_bwd,
                  make_opts)

FORMATS = {"e4m3": 0, "int8": 1}
DTYPES = {torch.bfloat16: 0, torch.float32: 1}
BLOCK = 32

_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _call(device, fn, *args):
    """fn(*args, stream) on ``device`` and its current stream.  Small calls
    last a few microseconds, as long as the marshalling around them: the
    stream handle is taken without a Stream object, and the device is switched
    only if it is not the current one."""
    i = device.index
    if i == _current_device():
        status = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            status = fn(*args, _raw_stream(i))
    if status:
        check(status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _opts(solver, max_iters, tol, warm_sweeps):
    """Solver options, None (the call's defaults) where nothing is chosen."""
    if solver == "newton" and max_iters is None and tol is None and warm_sweeps is None:
        return None
    return make_opts(solver, max_iters, tol, warm_sweeps)


def _format(format):
    if format not in FORMATS:
        raise ValueError(f"format must be one of {sorted(FORMATS)}")
    return FORMATS[format]


def _values(t, name):
    """A bf16 or fp32 tensor; returns the ABI's dtype code."""
    if isinstance(t, torch.Tensor) and t.dtype not in DTYPES:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    _need(t, name, getattr(t, "dtype", None))
    return DTYPES[t.dtype]


def _dtype(dtype):
    if dtype not in DTYPES:
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    return DTYPES[dtype]


def _scale_shape(shape):
    return tuple(shape[:-1]) + (-(-shape[-1] // BLOCK),)


def _pair(pair, name, shape, device):
    """A caller's (codes, scales) of an 8-bit checkpoint of ``shape``, both
    checked, or new ones if ``pair`` is None."""
    codes, scales = (None, None) if pair is None else pair
    return (_out(codes, f"{name} codes", torch.uint8, tuple(shape), device),
            _out(scales, f"{name} scales", torch.uint8, _scale_shape(shape), device))


def _given(pair, name, shape, device):
    """A checkpoint that a call reads."""
    codes, scales = pair
    if codes is None or scales is None:
        raise TypeError(f"{name} must be a (codes, scales) pair of tensors")
    return _pair(pair, name, shape, device)


def ckpt_pack(x: torch.Tensor, *, format="e4m3", out=None):
    """The 8-bit checkpoint (codes, scales) of x [..., C], bf16 or fp32, C a
    multiple of 8: blocks of 32 along the last axis.  ``out`` may be a
    previous pair."""
    fmt, dt = _format(format), _values(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be [..., C]")
    C = x.shape[-1]
    codes, scales = _pair(out, "out", x.shape, x.device)
    _call(x.device, lib().mhc_ckpt_pack, _ptr(x), dt, _ptr(codes), _ptr(scales),
          x.numel() // max(C, 1), C, fmt)
    return codes, scales


def ckpt_unpack(codes: torch.Tensor, scales: torch.Tensor, *, format="e4m3",
                dtype=torch.bfloat16, out=None):
    """The values a checkpoint stands for, as bf16 or fp32 (exact in both)."""
    fmt, dt = _format(format), _dtype(dtype)
    _need(codes, "codes", torch.uint8)
    if codes.dim() < 1:
        raise ValueError("codes must be [..., C]")
    _given((codes, scales), "checkpoint", codes.shape, codes.device)
    C = codes.shape[-1]
    x = _out(out, "out", dtype, codes.shape, codes.device)
    _call(codes.device, lib().mhc_ckpt_unpack, _ptr(codes), _ptr(scales), _ptr(x), dt,
          codes.numel() // max(C, 1), C, fmt)
    return x


def _mix_args(x_shape, device, H, name="H"):
    T, n, _ = x_shape
    _need(H, name, torch.float32)
    if tuple(H.shape) != (T, n, n) or H.device != device:
        raise ValueError(f"{name} must be [{T}, {n}, {n}] on {device}, got {tuple(H.shape)} on {H.device}")


def stream_mix_ckpt(x: torch.Tensor, H: torch.Tensor = None, *, logits: torch.Tensor = None,
                    format="e4m3", out=None, return_H=False, H_out=None, ckpt=None,
                    solver="newton", max_iters=None, tol=None, warm_sweeps=None):
    """``stream_mix`` that also writes x's checkpoint in the same pass.
    Returns (out, ckpt), or (out, H, ckpt) with ``return_H``; out and H are
    stream_mix's bit for bit, ckpt = (codes [T,4,C], scales)."""
    fmt = _format(format)
    _need(x, "x", torch.bfloat16)
    if x.dim() != 3:
        raise ValueError("x must be [T, n, C]")
    T, n, C = x.shape
    if (H is None) == (logits is None):
        raise ValueError("pass exactly one of H or logits")
    src = H if H is not None else logits
    _mix_args(x.shape, x.device, src, "H" if H is not None else "logits")
    y = _out(out, "out", torch.bfloat16, x.shape, x.device)
    if H_out is not None and not (logits is not None and return_H):
        raise ValueError("H_out needs logits and return_H")
    if logits is not None and return_H:
        H_out = _out(H_out, "H_out", torch.float32, logits.shape, x.device)
    elif return_H:
        H_out = H
    codes, scales = _pair(ckpt, "ckpt", x.shape, x.device)
    # a NULL proj means "H is given", so the projecting form always passes options
    o = make_opts(solver, max_iters, tol, warm_sweeps) if logits is not None else None
    _call(x.device, lib().mhc_stream_mix_ckpt, _ptr(x), _ptr(src),
          _ptr(H_out) if logits is not None else None, _ptr(y), _ptr(codes), _ptr(scales), T, n, C,
          fmt, ctypes.byref(o) if o is not None else None)
    return (y, H_out, (codes, scales)) if return_H else (y, (codes, scales))


def stream_mix_bwd_ckpt(ckpt, H: torch.Tensor, grad_out: torch.Tensor, *, format="e4m3", out=None):
    """``stream_mix_bwd`` with x read from its checkpoint: (grad_x bf16
    [T,4,C], grad_H fp32 [T,4,4]); ``out`` may be a preallocated pair."""
    fmt = _format(format)
    _need(grad_out, "grad_out", torch.bfloat16)
    if grad_out.dim() != 3:
        raise ValueError("grad_out must be [T, n, C]")
    T, n, C = grad_out.shape
    dev = grad_out.device
    codes, scales = _given(ckpt, "ckpt", grad_out.shape, dev)
    _mix_args(grad_out.shape, dev, H)
    gx, gH = (None, None) if out is None else out
    gx = _out(gx, "grad_x", torch.bfloat16, grad_out.shape, dev)
    gH = _out(gH, "grad_H", torch.float32, H.shape, dev)
    _call(dev, lib().mhc_stream_mix_bwd_ckpt, _ptr(codes), _ptr(scales), _ptr(H),
          _ptr(grad_out), _ptr(gx), _ptr(gH), T, n, C, fmt)
    return gx, gH


class ProjectedMix(torch.autograd.Function):
    """y = mix(projection(logits), x) with x kept for the backward as an 8-bit
    checkpoint (see projected_mix)."""

    @staticmethod
    def forward(ctx, x, logits, format, opts):
        x, logits = x.contiguous(), logits.contiguous()
        y, H, (codes, scales) = stream_mix_ckpt(x, logits=logits, return_H=True, format=format,
                                                **opts)
        ctx.format = format
        ctx.save_for_backward(codes, scales, H)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        codes, scales, H = ctx.saved_tensors
        gx, gH = stream_mix_bwd_ckpt((codes, scales), H, grad_y.contiguous(), format=ctx.format)
        return gx, birkhoff_bwd(H, gH, out=gH), None, None


def projected_mix(x, logits, *, format="e4m3", **opts):
    """Differentiable stream mix of x [T,4,C] bf16 by the projection of logits
    [T,4,4] fp32.  Keeps H and an 8-bit checkpoint of x; the gradient for the
    logits is that of the checkpointed x.  ``opts`` are the solver's."""
    return ProjectedMix.apply(x, logits, format, opts)


def _ckpt_args(ckpt, T, n, C, device, format, new):
    """(mhc_layer_ckpt, dict of pairs) of a layer's checkpoints, allocated
    where ``new`` and not given."""
    get = _pair if new else _given
    ckpt = {} if ckpt is None else ckpt
    x = get(ckpt.get("x") if new else ckpt["x"], "ckpt x", (T, n, C), device)
    f = get(ckpt.get("f") if new else ckpt["f"], "ckpt f", (T, C), device)
    k = LayerCkpt()
    k.format = _format(format)
    k.x_codes, k.x_scales = x[0].data_ptr(), x[1].data_ptr()
    k.f_codes, k.f_scales = f[0].data_ptr(), f[1].data_ptr()
    return k, dict(x=x, f=f)


def layer_fwd_ckpt(x, W, f, *, format="e4m3", eps=1e-6, solver="newton", max_iters=None, tol=None,
                   warm_sweeps=None, out=None, ckpt=None):
    """``layer_fwd`` that also writes the checkpoints of x and f.  Returns
    (forward dict, dict(x=(codes, scales), f=(codes, scales))); the forward's
    outputs are layer_fwd's bit for bit.  Only the checkpoints and the
    forward's rms, logits and maps are needed by layer_bwd_ckpt."""
    a = _layer_args(x, W, f, eps, _opts(solver, max_iters, tol, warm_sweeps))
    T, n, C = x.shape
    dev = x.device
    k, ckpt = _ckpt_args(ckpt, T, n, C, dev, format, True)
    out = _dict_out(out, _fwd_shapes(T, n, C), dev)
    for name, t in out.items():
        setattr(a, name, t.data_ptr())
    _call(dev, lib().mhc_layer_fwd_ckpt, ctypes.byref(a), ctypes.byref(k))
    return out, ckpt


def layer_ckpt_workspace(T, C, device, n=4):
    """Workspace of layer_bwd_ckpt for this shape (kept between calls by a
    training loop; calls that overlap in time need one each)."""
    nbytes = lib().mhc_layer_ckpt_workspace_bytes(T, n, C)
    if nbytes < 0:
        raise ValueError("invalid layer shape")
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def layer_bwd_ckpt(ckpt, W, fwd, grad_x_out, grad_u, *, format="e4m3", workspace=None, out=None):
    """``layer_bwd`` from the checkpoints of x and f (layer_fwd_ckpt's) and
    the forward's rms, logits, H_pre, H_post and H_res.  Returns dict(grad_x,
    grad_f, grad_W, grad_logits)."""
    _need(grad_x_out, "grad_x_out", torch.bfloat16)
    if grad_x_out.dim() != 3:
        raise ValueError("grad_x_out must be [T, n, C]")
    T, n, C = grad_x_out.shape
    dev = grad_x_out.device
    k, _ = _ckpt_args(ckpt, T, n, C, dev, format, False)
    _need(grad_u, "grad_u", torch.bfloat16)
    if tuple(grad_u.shape) != (T, C) or grad_u.device != dev:
        raise ValueError(f"grad_u must be [{T}, {C}] on {dev}, got {tuple(grad_u.shape)} on {grad_u.device}")
    # x and f enter only as shapes here: the checkpoints stand in for them
    a = _layer_args(grad_x_out, W, grad_u, 1e-6, None)
    a.x = a.f = None
    for name, (sh, dt) in _fwd_shapes(T, n, C).items():
        if name in ("u", "x_out"):
            continue
        t = fwd[name]
        _need(t, name, dt)
        if tuple(t.shape) != sh or t.device != dev:
            raise ValueError(f"{name} must be {sh} on {dev}, got {tuple(t.shape)} on {t.device}")
        setattr(a, name, t.data_ptr())
    a.grad_x_out, a.grad_u = grad_x_out.data_ptr(), grad_u.data_ptr()
    out = _dict_out(out, _bwd_shapes(T, n, C), dev)
    for name, t in out.items():
        setattr(a, name, t.data_ptr())
    if workspace is None:
        workspace = layer_ckpt_workspace(T, C, dev, n)
    _need(workspace, "workspace", torch.uint8)
    if workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}, got {workspace.device}")
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    if T == 0:
        out["grad_W"].zero_()  # a sum over no tokens; the call enqueues nothing
    _call(dev, lib().mhc_layer_bwd_ckpt, ctypes.byref(a), ctypes.byref(k))
    return out


# ---------------------------------------------------------------------------
# 4 bits
# ---------------------------------------------------------------------------

def mx4_quantize(x: torch.Tensor, *, transpose=False, out=None):
    """x [R, C] bf16 or fp32 to MXFP4 (codes [R, C/2], scales [R, C/32]),
    blocks of 32 along the rows (C a multiple of 32); with ``transpose`` the
    quantised transpose (codes [C, R/2], scales [C, R/32]), blocks along the
    columns (R a multiple of 32, C of 8)."""
    dt = _values(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [R, C]")
    R, C = x.shape
    rows, cols = (C, R) if transpose else (R, C)
    if cols % BLOCK:
        raise ValueError(f"the quantised axis must be a multiple of {BLOCK}, got {cols}")
    codes, scales = (None, None) if out is None else out
    codes = _out(codes, "codes", torch.uint8, (rows, cols // 2), x.device)
    scales = _out(scales, "scales", torch.uint8, (rows, cols // BLOCK), x.device)
    _call(x.device, lib().mhc_mx4_quantize, _ptr(x), dt, _ptr(codes), _ptr(scales), R, C,
          int(bool(transpose)))
    return codes, scales


def _mx4_given(pair, name):
    """(codes, scales, rows, columns) of a quantised matrix."""
    codes, scales = pair
    _need(codes, f"{name} codes", torch.uint8)
    if codes.dim() != 2 or codes.shape[1] % (BLOCK // 2):
        raise ValueError(f"{name} codes must be [R, C/2] with C a multiple of {BLOCK}")
    R, C = codes.shape[0], 2 * codes.shape[1]
    _need(scales, f"{name} scales", torch.uint8)
    if tuple(scales.shape) != (R, C // BLOCK) or scales.device != codes.device:
        raise ValueError(f"{name} scales must be [{R}, {C // BLOCK}] on {codes.device}, got "
                         f"{tuple(scales.shape)} on {scales.device}")
    return codes, scales, R, C


def mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, *, dtype=torch.bfloat16, out=None):
    """The values of a quantised matrix, [R, C] bf16 or fp32."""
    dt = _dtype(dtype)
    codes, scales, R, C = _mx4_given((codes, scales), "quantised")
    x = _out(out, "out", dtype, (R, C), codes.device)
    _call(codes.device, lib().mhc_mx4_dequantize, _ptr(codes), _ptr(scales), _ptr(x), dt, R, C)
    return x


def mx4_matmul(a, b, *, out_dtype=torch.bfloat16, out=None):
    """a b^T [M, N] for MXFP4 b = (codes, scales) [N, K] and a either such a
    pair [M, K] or a bf16 / fp32 tensor [M, K], which is quantised as
    mx4_quantize does.  N is a multiple of 8, K of 32; the sum is fp32."""
    od = _dtype(out_dtype)
    bc, bs, N, K = _mx4_given(b, "b")
    dev = bc.device
    if isinstance(a, torch.Tensor):
        ad = _values(a, "a")
        if a.dim() != 2 or a.shape[1] != K or a.device != dev:
            raise ValueError(f"a must be [M, {K}] on {dev}, got {tuple(a.shape)} on {a.device}")
        M = a.shape[0]
        y = _out(out, "out", out_dtype, (M, N), dev)
        need = lib().mhc_mx4_matmul_values_workspace_bytes(M, N, K)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
        _call(dev, lib().mhc_mx4_matmul_values, _ptr(a), ad, _ptr(bc), _ptr(bs), _ptr(y), od, M, N,
              K, _ptr(ws), max(need, 0))
        return y
    ac, as_, M, Ka = _mx4_given(a, "a")
    if Ka != K or ac.device != dev:
        raise ValueError(f"a must be [M, {K}] on {dev}, got [{M}, {Ka}] on {ac.device}")
    y = _out(out, "out", out_dtype, (M, N), dev)
    _call(dev, lib().mhc_mx4_matmul, _ptr(ac), _ptr(as_), _ptr(bc), _ptr(bs), _ptr(y), od, M, N,
          K)
    return y


def mx4_write_back(a, b, x, H_post, H_res, *, out=None, f_out=None):
    """x_out[t,i] = H_post[t,i] (a b^T)[t] + sum_j H_res[t,i,j] x[t,j] for
    MXFP4 pairs a [T, K] and b [C, K], x [T,4,C] bf16: the layer function's
    last product with the layer's write-back in its epilogue.  ``f_out``
    [T, C] bf16, if given, also receives a b^T."""
    _need(x, "x", torch.bfloat16)
    if x.dim() != 3:
        raise ValueError("x must be [T, n, C]")
    T, n, C = x.shape
    dev = x.device
    ac, as_, M, K = _mx4_given(a, "a")
    bc, bs, N, Kb = _mx4_given(b, "b")
    if M != T or N != C or K != Kb or ac.device != dev or bc.device != dev:
        raise ValueError(f"a and b must be [{T}, K] and [{C}, K] on {dev}, got [{M}, {K}] on "
                         f"{ac.device} and [{N}, {Kb}] on {bc.device}")
    for t, name, shape in ((H_post, "H_post", (T, n)), (H_res, "H_res", (T, n, n))):
        _need(t, name, torch.float32)
        if tuple(t.shape) != shape or t.device != dev:
            raise ValueError(f"{name} must be {shape} on {dev}, got {tuple(t.shape)} on {t.device}")
    y = _out(out, "out", torch.bfloat16, x.shape, dev)
    if f_out is not None:
        f_out = _out(f_out, "f_out", torch.bfloat16, (T, C), dev)
    _call(dev, lib().mhc_mx4_write_back, _ptr(ac), _ptr(as_), _ptr(bc), _ptr(bs), _ptr(x),
          _ptr(H_post), _ptr(H_res), _ptr(y), _ptr(f_out), T, n, C, K)
    return y


def layer_read(x, W, *, mx4=False, keep_u=False, eps=1e-6, solver="newton", max_iters=None,
               tol=None, warm_sweeps=None, out=None):
    """The read half of the layer step: dict(rms, logits, H_pre, H_post,
    H_res, u) from x [T,4,C] and W [24,4C] bf16.  With ``mx4`` u is the MXFP4
    pair of the bf16 u (which ``keep_u`` also returns, as "u_values").
    ``out`` may be a previous result dict."""
    o = _opts(solver, max_iters, tol, warm_sweeps)
    _need(x, "x", torch.bfloat16)
    if x.dim() != 3:
        raise ValueError("x must be [T, n, C]")
    T, n, C = x.shape
    dev = x.device
    _need(W, "W", torch.bfloat16)
    if tuple(W.shape) != (n * n + 2 * n, n * C) or W.device != dev:
        raise ValueError(f"W must be [n*n+2n, n*C] on {dev}, got {tuple(W.shape)} on {W.device}")
    out = {} if out is None else out
    a = LayerArgs()
    a.T, a.n, a.C, a.eps = T, n, C, float(eps)
    a.proj = ctypes.pointer(o) if o is not None else None
    a.x, a.W = x.data_ptr(), W.data_ptr()
    shapes = {k: v for k, v in _fwd_shapes(T, n, C).items() if k not in ("u", "x_out")}
    r = _dict_out(out, shapes, dev)
    for name, t in r.items():
        setattr(a, name, t.data_ptr())
    codes = scales = None
    if mx4:
        codes, scales = (None, None) if out.get("u") is None else out["u"]
        codes = _out(codes, "u codes", torch.uint8, (T, C // 2), dev)
        scales = _out(scales, "u scales", torch.uint8, (T, C // BLOCK), dev)
        r["u"] = (codes, scales)
    if keep_u or not mx4:
        key = "u_values" if mx4 else "u"
        r[key] = _out(out.get(key), key, torch.bfloat16, (T, C), dev)
        a.u = r[key].data_ptr()
    need = lib().mhc_layer_read_workspace_bytes(T, n, C)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    a.workspace, a.workspace_bytes = (ws.data_ptr() if ws is not None else None), max(need, 0)
    _call(dev, lib().mhc_layer_read, ctypes.byref(a), _ptr(codes), _ptr(scales))
    return r


class Mx4Linear(torch.autograd.Function):
    """y = x w^T with every product on MXFP4 operands (see mx4_linear)."""

    @staticmethod
    def forward(ctx, x, w, format):
        x, w = x.contiguous(), w.contiguous()
        y = mx4_matmul(x, mx4_quantize(w), out_dtype=x.dtype)
        codes, scales = ckpt_pack(x, format=format)
        ctx.format, ctx.dtype = format, x.dtype
        ctx.save_for_backward(codes, scales, w)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        codes, scales, w = ctx.saved_tensors
        gy = gy.contiguous()
        gx = gw = None
        if ctx.needs_input_grad[0]:
            gx = mx4_matmul(gy, mx4_quantize(w, transpose=True), out_dtype=ctx.dtype)
        if ctx.needs_input_grad[1] and gy.shape[0] == 0:
            gw = torch.zeros_like(w)
        elif ctx.needs_input_grad[1]:
            x = ckpt_unpack(codes, scales, format=ctx.format, dtype=ctx.dtype)
            gw = mx4_matmul(mx4_quantize(gy, transpose=True), mx4_quantize(x, transpose=True),
                            out_dtype=w.dtype)
        return gx, gw, None


def mx4_linear(x, w, *, format="e4m3"):
    """Differentiable y = x w^T [M, N] for x [M, K], w [N, K] bf16 or fp32 (M,
    N and K multiples of 32).  Each of the three products takes both operands
    in MXFP4, quantised along the axis it sums over: y = q(x) q(w)^T,
    grad_x = q(gy) q(w^T)^T, grad_w = q(gy^T) q(xhat^T)^T.  x is kept for the
    backward as an 8-bit checkpoint (xhat), w as it is."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must be [M, K] and [N, K]")
    if any(s % BLOCK for s in (*x.shape, *w.shape)):
        raise ValueError(f"M, N and K must be multiples of {BLOCK}, got x {tuple(x.shape)} and "
                         f"w {tuple(w.shape)}")
    return Mx4Linear.apply(x, w, format)
