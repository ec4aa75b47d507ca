"""Float64 CPU oracle for blocks of 32 values with a shared power-of-two scale.

TEST INFRASTRUCTURE ONLY (imported by tests/; never by the product package).

The formats, as include/mhc.h defines them: a block of 32 consecutive values of
a row has a scale byte s standing for 2^(s - 127), the smallest power of two
with max|block| <= M 2^(s - 127), clamped to [lo, 254]; s = 255 and zero codes
if the block holds an infinity or a NaN.  A value's code is that of the nearest
element of the table of the format's values times the scale, ties to the even
code.  Elements are looked up in the written-out table, by the definition of
the format, not by bit arithmetic.  Elements that would stand for 2^128 or
more (no fp32 or bf16 number) are not used.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def _float_table(mantissa_bits, emin, largest):
    """Non-negative values of a small float format, in code order."""
    out, code = [], 0
    while True:
        e, m = divmod(code, 1 << mantissa_bits)
        if e == 0:
            v = m * 2.0 ** (emin - mantissa_bits)
        else:
            v = (1 + m / (1 << mantissa_bits)) * 2.0 ** (emin + e - 1)
        if v > largest:
            return np.array(out)
        out.append(v)
        code += 1


TABLES = {
    "e4m3": _float_table(3, -6, 448.0),
    "int8": np.arange(128) / 64.0,
    "e2m1": _float_table(1, 0, 6.0),
}
LARGEST = {k: t[-1] for k, t in TABLES.items()}
LO = {"e4m3": 10, "int8": 7, "e2m1": 2}


def _nearest(a, table):
    """Index of the entry of `table` nearest to each a >= 0, ties to even."""
    mid = (table[1:] + table[:-1]) / 2
    i = np.searchsorted(mid, a)  # number of midpoints below a
    at = np.minimum(i, len(mid) - 1)
    return i + ((i < len(mid)) & (mid[at] == a) & (i % 2 == 1))


def quantise(x, fmt):
    """(codes, scales, values) of x [..., C] along its last axis: codes one
    per value (uint8: sign bit and index, or two's complement for int8),
    scales uint8 [..., ceil(C/32)], values float64."""
    x = np.asarray(x, dtype=np.float64)
    C = x.shape[-1]
    v = np.pad(x.reshape(-1, C), ((0, 0), (0, -C % BLOCK))).reshape(-1, -(-C // BLOCK), BLOCK)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    amax = np.abs(v).max(-1)
    e = np.full(amax.shape, LO[fmt] - 127)
    nz = amax > 0
    e[nz] = np.ceil(np.log2(amax[nz] / LARGEST[fmt])).astype(int)
    # log2 is rounded: settle each exponent by the definition itself
    e = np.where(amax > LARGEST[fmt] * 2.0 ** e, e + 1, e)
    e = np.where(nz & (amax <= LARGEST[fmt] * 2.0 ** (e - 1.0)), e - 1, e)
    s = np.clip(e + 127, LO[fmt], 254)
    scale = 2.0 ** (s - 127.0)
    i = _nearest(np.abs(v) / scale[..., None], TABLES[fmt])
    i = np.where(TABLES[fmt][i] * scale[..., None] >= 2.0 ** 128, i - 1, i)
    neg = np.signbit(v)
    values = np.where(neg, -1.0, 1.0) * TABLES[fmt][i] * scale[..., None]
    if fmt == "int8":
        codes = np.where(neg, -i, i) & 0xFF
    else:
        codes = i | np.where(neg, sign_bit(fmt), 0)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    values = np.where(bad[..., None], np.nan, values)
    s = np.where(bad, 255, s).astype(np.uint8)
    shape = x.shape
    cut = lambda t: t.reshape(len(v), -1)[:, :C].reshape(shape)
    return cut(codes), s.reshape(shape[:-1] + (-1,)), cut(values)


def sign_bit(fmt):
    """The sign bit of a float format's code."""
    return 0x80 if fmt == "e4m3" else 8


def pack4(codes):
    """4-bit codes [R, C] to bytes [R, C/2], the even one in the low half."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def values4(packed, scales):
    """Values of MXFP4 bytes [R, C/2] with any scale bytes [R, C/32]."""
    c = np.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1)
    v = np.where(c > 7, -1.0, 1.0) * TABLES["e2m1"][c & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, BLOCK, axis=1)


def layer_bwd(xhat, W, fhat, dx_out, du, fwd):
    """The layer backward with x and f replaced by what their checkpoints
    stand for, and the forward's rms, logits and maps taken as given.  Differs
    from oracle.layer_bwd in the RMSNorm term, whose <dl W, x / r> is
    <dl, logits> with the forward's logits."""
    from .birkhoff import birkhoff_project_bwd
    T, n, C = xhat.shape
    D = n * C
    Hp, Ho, Hr, r, lg = (np.asarray(fwd[k], np.float64) for k in
                         ("H_pre", "H_post", "H_res", "rms", "logits"))
    d_pre = np.einsum("tc,tjc->tj", du, xhat)
    d_post = np.einsum("tic,tc->ti", dx_out, fhat)
    d_res = np.einsum("tic,tjc->tij", dx_out, xhat)
    dl = np.concatenate([d_pre * Hp * (1 - Hp), d_post * Ho * (1 - Ho),
                         birkhoff_project_bwd(Hr, d_res).reshape(T, n * n)], axis=1)
    xn = xhat.reshape(T, D) / r[:, None]
    dn = (dl @ W - xn * ((dl * lg).sum(1) / D)[:, None]) / r[:, None]
    dx = np.einsum("tij,tic->tjc", Hr, dx_out) + Hp[:, :, None] * du[:, None, :] + dn.reshape(T, n, C)
    return dict(dx=dx, dW=dl.T @ xn, df=np.einsum("ti,tic->tc", Ho, dx_out), dlogits=dl,
                d_res=d_res, d_pre=d_pre, d_post=d_post)
