"""Python entry points over the checkpoint and 4-bit calls of the C ABI.

Like ``ops``, these take CUDA (HIP) tensors, refuse what does not fit before
anything is enqueued, run on the tensors' device and its current stream and
return the output tensors; all arithmetic runs in the gfx950 kernels.  The
marshalling itself is the extension module ``_binding`` (csrc/binding.cpp):
through ctypes it would take longer than the smallest calls.

A packed tensor is a pair ``(codes, scales)`` of uint8 tensors: one scale byte
s, standing for 2^(s - 127), for each 32 consecutive values of a row.  8-bit
checkpoints have ``format`` "e4m3" (8-bit floating point) or "int8" (multiples
of 1/64 of the scale) and codes of the values' shape.  4-bit (MXFP4) codes hold
two values a byte, the even one in the low half.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._lib import binding, check
from .ops import SOLVERS, birkhoff_bwd

FORMATS = {"e4m3": 0, "int8": 1}
DTYPES = {torch.bfloat16: 0, torch.float32: 1}
BLOCK = 32
_MAPS = ("rms", "logits", "H_pre", "H_post", "H_res")
_NO_PAIR = (None, None)


def _format(format):
    if format not in FORMATS:
        raise ValueError(f"format must be one of {sorted(FORMATS)}")
    return FORMATS[format]


def _dtype(dtype):
    if dtype not in DTYPES:
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    return DTYPES[dtype]


def _opts(solver, max_iters, tol, warm_sweeps):
    """Solver options; -1 (tol: any negative) stands for the default."""
    if solver not in SOLVERS:
        raise ValueError(f"solver must be one of {sorted(SOLVERS)}")
    if tol is not None and not tol >= 0:
        raise ValueError(f"tol must be in [0, 1], got {tol}")
    return (SOLVERS[solver], -1 if max_iters is None else int(max_iters),
            -1.0 if tol is None else float(tol), -1 if warm_sweeps is None else int(warm_sweeps))


def ckpt_pack(x: torch.Tensor, *, format="e4m3", out=None):
    """The 8-bit checkpoint (codes, scales) of x [..., C], bf16 or fp32, C a
    multiple of 8: blocks of 32 along the last axis.  ``out`` may be a
    previous pair."""
    codes, scales = _NO_PAIR if out is None else out
    status, codes, scales = binding().ckpt_pack(x, _format(format), codes, scales)
    if status:
        check(status)
    return codes, scales


def ckpt_unpack(codes: torch.Tensor, scales: torch.Tensor, *, format="e4m3",
                dtype=torch.bfloat16, out=None):
    """The values a checkpoint stands for, as bf16 or fp32 (exact in both)."""
    status, x = binding().ckpt_unpack(codes, scales, _format(format), _dtype(dtype), out)
    if status:
        check(status)
    return x


def stream_mix_ckpt(x: torch.Tensor, H: torch.Tensor = None, *, logits: torch.Tensor = None,
                    format="e4m3", out=None, return_H=False, H_out=None, ckpt=None,
                    solver="newton", max_iters=None, tol=None, warm_sweeps=None):
    """``stream_mix`` that also writes x's checkpoint in the same pass.
    Returns (out, ckpt), or (out, H, ckpt) with ``return_H``; out and H are
    stream_mix's bit for bit, ckpt = (codes [T,4,C], scales)."""
    if (H is None) == (logits is None):
        raise ValueError("pass exactly one of H or logits")
    if H_out is not None and not (logits is not None and return_H):
        raise ValueError("H_out needs logits and return_H")
    codes, scales = _NO_PAIR if ckpt is None else ckpt
    opts = _opts(solver, max_iters, tol, warm_sweeps) if H is None else None
    status, y, H_new, codes, scales = binding().stream_mix_ckpt(
        x, logits if H is None else H, _format(format), opts, return_H, out, H_out, codes, scales)
    if status:
        check(status)
    if return_H:
        return y, H_new if H is None else H, (codes, scales)
    return y, (codes, scales)


def stream_mix_bwd_ckpt(ckpt, H: torch.Tensor, grad_out: torch.Tensor, *, format="e4m3", out=None):
    """``stream_mix_bwd`` with x read from its checkpoint: (grad_x bf16
    [T,4,C], grad_H fp32 [T,4,4]); ``out`` may be a preallocated pair."""
    codes, scales = ckpt
    gx, gH = _NO_PAIR if out is None else out
    status, gx, gH = binding().stream_mix_bwd_ckpt(codes, scales, H, grad_out, _format(format), gx,
                                                   gH)
    if status:
        check(status)
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
        binding().stays_in_capture()
        codes, scales, H = ctx.saved_tensors
        gx, gH = stream_mix_bwd_ckpt((codes, scales), H, grad_y.contiguous(), format=ctx.format)
        return gx, birkhoff_bwd(H, gH, out=gH), None, None


def projected_mix(x, logits, *, format="e4m3", **opts):
    """Differentiable stream mix of x [T,4,C] bf16 by the projection of logits
    [T,4,4] fp32.  Keeps H and an 8-bit checkpoint of x; the gradient for the
    logits is that of the checkpointed x.  ``opts`` are the solver's.  A
    captured backward raises where it would reach an eager graph on the default
    stream, at x or logits or behind their casts and views."""
    return ProjectedMix.apply(x, logits, format, opts)


def layer_fwd_ckpt(x, W, f, *, format="e4m3", eps=1e-6, solver="newton", max_iters=None, tol=None,
                   warm_sweeps=None, out=None, ckpt=None):
    """``layer_fwd`` that also writes the checkpoints of x and f.  Returns
    (forward dict, dict(x=(codes, scales), f=(codes, scales))).  The maps are
    layer_read's bit for bit; with more than 2048 tokens (8192 where C is
    2048 or more) all of the forward is layer_fwd's.  Only the checkpoints and
    the forward's rms, logits and maps are needed by layer_bwd_ckpt.  ``out`` and ``ckpt`` may be previous
    results."""
    out, ckpt = out or {}, ckpt or {}
    status, maps, (u, x_out), k = binding().layer_fwd_ckpt(
        x, W, f, _format(format), eps, _opts(solver, max_iters, tol, warm_sweeps),
        [out.get(m) for m in _MAPS] if out else [], [out.get("u"), out.get("x_out")],
        [*ckpt.get("x", _NO_PAIR), *ckpt.get("f", _NO_PAIR)])
    if status:
        check(status)
    return (dict(zip(_MAPS, maps), u=u, x_out=x_out),
            dict(x=(k[0], k[1]), f=(k[2], k[3])))


def layer_ckpt_workspace(T, C, device, n=4):
    """Workspace of layer_bwd_ckpt for this shape (kept between calls by a
    training loop; calls that overlap in time need one each)."""
    from ._lib import lib
    nbytes = lib().mhc_layer_ckpt_workspace_bytes(T, n, C)
    if nbytes < 0:
        raise ValueError("invalid layer shape")
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def layer_bwd_ckpt(ckpt, W, fwd, grad_x_out, grad_u, *, format="e4m3", workspace=None, out=None):
    """``layer_bwd`` from the checkpoints of x and f (layer_fwd_ckpt's) and
    the forward's rms, logits, H_pre, H_post and H_res.  Returns dict(grad_x,
    grad_f, grad_W, grad_logits)."""
    names = ("grad_x", "grad_f", "grad_W", "grad_logits")
    out = out or {}
    status, grads = binding().layer_bwd_ckpt(
        [*ckpt["x"], *ckpt["f"]], W, [fwd[m] for m in _MAPS], grad_x_out, grad_u, _format(format),
        workspace, [out.get(k) for k in names])
    if status:
        check(status)
    grads = dict(zip(names, grads))
    if grad_x_out.shape[0] == 0:
        grads["grad_W"].zero_()  # a sum over no tokens; the call enqueues nothing
    return grads


def layer_read(x, W, *, mx4=False, keep_u=False, eps=1e-6, solver="newton", max_iters=None,
               tol=None, warm_sweeps=None, out=None):
    """The read half of the layer step: dict(rms, logits, H_pre, H_post,
    H_res, u) from x [T,4,C] and W [24,4C] bf16.  With ``mx4`` u is the MXFP4
    pair of the bf16 u (which ``keep_u`` also returns, as "u_values").
    ``out`` may be a previous result dict."""
    out = out or {}
    codes, scales = (out.get("u") or _NO_PAIR) if mx4 else _NO_PAIR
    status, maps, u, codes, scales = binding().layer_read(
        x, W, mx4, keep_u or not mx4, eps, _opts(solver, max_iters, tol, warm_sweeps),
        [out.get(m) for m in _MAPS] if out else [], out.get("u_values" if mx4 else "u"), codes,
        scales)
    if status:
        check(status)
    r = dict(zip(_MAPS, maps))
    r["u"] = (codes, scales) if mx4 else u
    if mx4 and keep_u:
        r["u_values"] = u
    return r


# ---------------------------------------------------------------------------
# 4 bits
# ---------------------------------------------------------------------------

def mx4_quantize(x: torch.Tensor, *, transpose=False, out=None):
    """x [R, C] bf16 or fp32 to MXFP4 (codes [R, C/2], scales [R, C/32]),
    blocks of 32 along the rows (C a multiple of 32); with ``transpose`` the
    quantised transpose (codes [C, R/2], scales [C, R/32]), blocks along the
    columns (R a multiple of 32, C of 8)."""
    codes, scales = _NO_PAIR if out is None else out
    status, codes, scales = binding().mx4_quantize(x, transpose, codes, scales)
    if status:
        check(status)
    return codes, scales


def mx4_quantize_both(x: torch.Tensor):
    """mx4_quantize(x) and mx4_quantize(x, transpose=True) in one pass over x
    [R, C] bf16 or fp32, R and C multiples of 32."""
    status, codes, scales, t_codes, t_scales = binding().mx4_quantize_both(x)
    if status:
        check(status)
    return (codes, scales), (t_codes, t_scales)


def mx4_quantize_ckpt(x: torch.Tensor, *, format="e4m3"):
    """mx4_quantize(x) and ckpt_pack(x, format=format) in one pass over x
    [R, C] bf16 or fp32, C a multiple of 32."""
    status, codes, scales, c_codes, c_scales = binding().mx4_quantize_ckpt(x, _format(format))
    if status:
        check(status)
    return (codes, scales), (c_codes, c_scales)


def mx4_requantize(codes: torch.Tensor, scales: torch.Tensor, *, format="e4m3"):
    """mx4_quantize(ckpt_unpack(codes, scales), transpose=True) in one pass:
    the quantised transpose of a checkpoint [R, C], R and C multiples of 32."""
    status, q_codes, q_scales = binding().mx4_requantize(codes, scales, _format(format))
    if status:
        check(status)
    return q_codes, q_scales


def mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, *, dtype=torch.bfloat16, out=None):
    """The values of a quantised matrix, [R, C] bf16 or fp32."""
    status, x = binding().mx4_dequantize(codes, scales, _dtype(dtype), out)
    if status:
        check(status)
    return x


def mx4_matmul(a, b, *, out_dtype=torch.bfloat16, out=None):
    """a b^T [M, N] for MXFP4 b = (codes, scales) [N, K] and a either such a
    pair [M, K] or a bf16 / fp32 tensor [M, K], which is quantised as
    mx4_quantize does.  N is a multiple of 8, K of 32; the sum is fp32."""
    bc, bs = b
    if isinstance(a, torch.Tensor):
        status, y = binding().mx4_matmul_values(a, bc, bs, _dtype(out_dtype), out)
    else:
        ac, as_ = a
        status, y = binding().mx4_matmul(ac, as_, bc, bs, _dtype(out_dtype), out)
    if status:
        check(status)
    return y


def mx4_write_back(a, b, x, H_post, H_res, *, out=None, f_out=None):
    """x_out[t,i] = H_post[t,i] (a b^T)[t] + sum_j H_res[t,i,j] x[t,j] for
    MXFP4 pairs a [T, K] and b [C, K], x [T,4,C] bf16: the layer function's
    last product with the layer's write-back in its epilogue.  ``f_out``
    [T, C] bf16, if given, also receives a b^T."""
    (ac, as_), (bc, bs) = a, b
    status, y = binding().mx4_write_back(ac, as_, bc, bs, x, H_post, H_res, out, f_out)
    if status:
        check(status)
    return y


def mx4_linear(x, w, *, format="e4m3"):
    """Differentiable y = x w^T [M, N] for x [M, K], w [N, K] bf16 or fp32 (M,
    N and K multiples of 32).  Each of the three products takes both operands
    in MXFP4, quantised along the axis it sums over: y = q(x) q(w)^T,
    grad_x = q(gy) q(w^T)^T, grad_w = q(gy^T) q(xhat^T)^T.  x is kept for the
    backward as an 8-bit checkpoint (xhat), w as it is, whichever gradients are
    wanted; without any, mx4_matmul of a quantised w does less.  Differentiable once.
    A captured backward raises where it would reach an eager graph on the
    default stream, at w or x or behind their casts and views."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must be [M, K] and [N, K]")
    if any(s % BLOCK for s in (*x.shape, *w.shape)):
        raise ValueError(f"M, N and K must be multiples of {BLOCK}, got x {tuple(x.shape)} and "
                         f"w {tuple(w.shape)}")
    return binding().mx4_linear(x, w, _format(format))
