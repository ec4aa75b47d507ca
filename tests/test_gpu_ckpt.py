"""GPU parity of the 8-bit checkpoints, of the stream mix and the layer step
that use them, and of 4-bit quantisation, against the float64 oracle.

Codes and scales are compared bit for bit: dividing by a power of two is
exact, so there is one rounding and it is the definition's.

Bars of the computed outputs (a rounding is off by at most half a step: u =
2^-24 of the value in fp32, 2^-8 in bf16):
  grad_H      a sum of C products of exact values in fp32: each lane adds at
              most 8 ceil(C / 512) of them in a chain and the wave's sum adds 6
              levels, so |d| <= (8 ceil(C / 512) + 7) u sum|terms|
  grad_x (mix), out, u, x_out and the maps: bit for bit those of the plain
              calls, which have their own bars
  layer       the plain layer's bars (test_gpu_layer.py) with xhat, fhat in
              the place of x, f; grad_W tighter, see there
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import birkhoff_project, birkhoff_project_bwd, layer_bwd as o_layer_bwd, packed as K

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FMTS = ["e4m3", "int8"]


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def rand(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def hard_rows(R, C, seed, dtype):
    """Rows of widely different sizes, with ties, zeros, subnormals, the
    type's largest values and non-finite entries spread over them."""
    g = np.random.Generator(np.random.PCG64(seed))
    x = g.standard_normal((R, C)) * np.exp2(g.integers(-40, 40, (R, 1)))
    x *= np.exp2(g.integers(-6, 7, (R, C)))
    kind = np.arange(R) % 8
    x[kind == 1] = np.round(x[kind == 1] / np.abs(x[kind == 1]).max(initial=1) * 64) / 32  # ties
    x[kind == 2] *= 0.0
    x[kind == 3] = g.standard_normal((int((kind == 3).sum()), C)) * 1e-38
    x[kind == 4] = np.sign(g.standard_normal((int((kind == 4).sum()), C))) * 3.3e38
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    if R > 7:
        t[5, C // 2] = float("inf")
        t[6, 0] = float("nan")
        t[7, C - 1] = float("-inf")
    return t.cuda()


SHAPES = [(1, 8), (3, 40), (9, 32), (16, 1000), (129, 72), (64, 256), (1, 8192), (2051, 264), (1, 24)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,C", SHAPES)
def test_pack_and_unpack(gpu_lib, R, C, fmt, dtype):
    print(f"pack {R}x{C} {fmt} {dtype}", flush=True)
    x = hard_rows(R, C, 10 * R + C, dtype)
    # written into the head of longer buffers, whose tails must stay
    cb = torch.full((R + 3, C), 0x5A, dtype=torch.uint8, device="cuda")
    sb = torch.full((R + 3, -(-C // 32)), 0x5A, dtype=torch.uint8, device="cuda")
    codes, scales = gpu_lib.ckpt_pack(x, format=fmt, out=(cb[:R], sb[:R]))
    ref_c, ref_s, ref_v = K.quantise(f64(x) if dtype == torch.bfloat16 else x.cpu().numpy(), fmt)
    assert (scales.cpu().numpy() == ref_s).all()
    got = codes.cpu().numpy()
    if fmt == "e4m3":  # the sign of a zero is not part of the value
        same = (got == ref_c) | (((got | ref_c) & 0x7F) == 0)
    else:
        same = got == ref_c
    assert same.all(), np.argwhere(~same)[:4]
    for dt in (torch.bfloat16, torch.float32):
        vb = torch.full((R + 3, C), 7.0, dtype=dt, device="cuda")
        v = gpu_lib.ckpt_unpack(codes, scales, format=fmt, dtype=dt, out=vb[:R])
        assert np.array_equal(f64(v), ref_v, equal_nan=True)  # exact in both types
        assert bool((vb[R:] == 7.0).all())
    assert bool((cb[R:] == 0x5A).all()) and bool((sb[R:] == 0x5A).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("R,C", [(32, 32), (64, 96), (288, 160), (1, 64), (32, 8), (512, 72), (2080, 64),
                                 (7, 4096), (544, 4096)])
def test_mx4_quantize(gpu_lib, R, C, transpose, dtype):
    if (transpose and R % 32) or (not transpose and C % 32):
        with pytest.raises(ValueError):
            gpu_lib.mx4_quantize(torch.zeros(R, C, dtype=dtype, device="cuda"), transpose=transpose)
        return
    print(f"mx4 {R}x{C} transpose={transpose} {dtype}", flush=True)
    x = hard_rows(R, C, R + 7 * C, dtype)
    rows, cols = (C, R) if transpose else (R, C)
    cb = torch.full((rows + 3, cols // 2), 0x5A, dtype=torch.uint8, device="cuda")
    sb = torch.full((rows + 3, cols // 32), 0x5A, dtype=torch.uint8, device="cuda")
    codes, scales = gpu_lib.mx4_quantize(x, transpose=transpose, out=(cb[:rows], sb[:rows]))
    x64 = f64(x) if dtype == torch.bfloat16 else x.cpu().numpy().astype(np.float64)
    ref_c, ref_s, ref_v = K.quantise(x64.T if transpose else x64, "e2m1")
    assert (scales.cpu().numpy() == ref_s).all()
    got = codes.cpu().numpy()
    got = np.stack((got & 15, got >> 4), -1).reshape(rows, cols)
    assert ((got == ref_c) | (((got | ref_c) & 7) == 0)).all()
    for dt in (torch.bfloat16, torch.float32):
        assert np.array_equal(f64(gpu_lib.mx4_dequantize(codes, scales, dtype=dt)), ref_v, equal_nan=True)
    assert bool((cb[rows:] == 0x5A).all()) and bool((sb[rows:] == 0x5A).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(32, 32), (64, 96), (288, 160), (256, 64), (320, 1088), (2080, 64), (544, 4096)])
def test_mx4_joint_quantisation(gpu_lib, R, C, dtype):
    """What one pass writes twice is what two calls write, bit for bit, for
    values near the formats' limits, infinities and NaN too."""
    print(f"mx4 joint {R}x{C} {dtype}", flush=True)
    x = hard_rows(R, C, R + C, dtype)
    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(a, b))
    rows, cols = gpu_lib.mx4_quantize_both(x)
    assert same(rows, gpu_lib.mx4_quantize(x)) and same(cols, gpu_lib.mx4_quantize(x, transpose=True))
    for fmt in FMTS:
        q, ck = gpu_lib.mx4_quantize_ckpt(x, format=fmt)
        assert same(q, rows) and same(ck, gpu_lib.ckpt_pack(x, format=fmt))
        back = gpu_lib.ckpt_unpack(*ck, format=fmt, dtype=dtype)
        assert same(gpu_lib.mx4_requantize(*ck, format=fmt), gpu_lib.mx4_quantize(back, transpose=True))


def test_mx4_quantize_ckpt_any_rows(gpu_lib):
    for R in (1, 7, 33):
        x = rand((R, 96), R)
        q, ck = gpu_lib.mx4_quantize_ckpt(x, format="int8")
        for a, b in zip((*q, *ck), (*gpu_lib.mx4_quantize(x), *gpu_lib.ckpt_pack(x, format="int8"))):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):
        gpu_lib.mx4_quantize_both(rand((33, 64), 1))
    with pytest.raises(ValueError):
        gpu_lib.mx4_quantize_ckpt(rand((32, 40), 1))
    c, s = gpu_lib.ckpt_pack(rand((32, 64), 1))
    with pytest.raises(ValueError):
        gpu_lib.mx4_requantize(c, s[:31])


def test_dequantize_reads_any_scale_byte(gpu_lib):
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(0, 256, (256, 32), generator=g, dtype=torch.uint8)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 2)
    v = gpu_lib.mx4_dequantize(codes.cuda(), scales.cuda(), dtype=torch.float32)
    with np.errstate(over="ignore"):
        ref = K.values4(codes.numpy(), scales.numpy()).astype(np.float32)
    assert np.array_equal(v.cpu().numpy(), ref, equal_nan=True)


def test_pack_past_32_bit_offsets(gpu_lib):
    """More than 2^32 values: the last rows come out as the same rows alone."""
    R, C = (1 << 32) // 4096 + 40, 4096
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    tail = rand((64, C), 8)
    x[-64:] = tail
    codes, scales = gpu_lib.ckpt_pack(x, format="int8")
    c1, s1 = gpu_lib.ckpt_pack(tail, format="int8")
    assert torch.equal(codes[-64:], c1) and torch.equal(scales[-64:], s1)
    assert int(codes[:-64].max()) == 0
    del x
    back = gpu_lib.ckpt_unpack(codes, scales, format="int8")
    assert torch.equal(back[-64:], gpu_lib.ckpt_unpack(c1, s1, format="int8"))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,C", [(1, 8), (15, 64), (16, 200), (17, 4096), (100, 520), (241, 72), (4099, 136),
                                 (3, 5792), (2049, 520)])
def test_mix_ckpt(gpu_lib, T, C, fmt):
    print(f"mix ckpt T={T} C={C} {fmt}", flush=True)
    x, g = rand((T, 4, C), T + C), rand((T, 4, C), T + C + 1)
    logits = torch.from_numpy(W.logits_batch("normal2", T, T)).cuda()
    for kw in (dict(logits=logits, return_H=True), dict(logits=logits, return_H=True, solver="sinkhorn")):
        out, H, ckpt = gpu_lib.stream_mix_ckpt(x, format=fmt, **kw)
        out0, H0 = gpu_lib.stream_mix(x, **kw)
        assert torch.equal(out, out0) and torch.equal(H, H0)
    out2, ckpt2 = gpu_lib.stream_mix_ckpt(x, H, format=fmt)
    assert torch.equal(out2, gpu_lib.stream_mix(x, H))
    codes, scales = gpu_lib.ckpt_pack(x, format=fmt)
    for c in (ckpt, ckpt2):
        assert torch.equal(c[0], codes) and torch.equal(c[1], scales)
    gx, gH = gpu_lib.stream_mix_bwd_ckpt(ckpt, H, g, format=fmt)
    gx0, _ = gpu_lib.stream_mix_bwd(x, H, g)
    assert torch.equal(gx, gx0)
    xh, g64 = f64(gpu_lib.ckpt_unpack(codes, scales, format=fmt)), f64(g)
    ref = np.einsum("tic,tjc->tij", g64, xh)
    mag = np.einsum("tic,tjc->tij", np.abs(g64), np.abs(xh))
    err = np.abs(gH.cpu().numpy() - ref)
    assert (err <= (8 * -(-C // 512) + 7) * U * mag).all(), (err / np.maximum(mag, 1e-30)).max() / U


def test_mix_ckpt_writes_only_its_tokens(gpu_lib):
    T, C = 17, 200
    x, g, H = rand((T, 4, C), 1), rand((T, 4, C), 2), rand((T, 4, 4), 3, torch.float32)
    full = dict(out=torch.full((T + 2, 4, C), 9.0, dtype=torch.bfloat16, device="cuda"),
                codes=torch.full((T + 2, 4, C), 77, dtype=torch.uint8, device="cuda"),
                scales=torch.full((T + 2, 4, 7), 77, dtype=torch.uint8, device="cuda"),
                gx=torch.full((T + 2, 4, C), 9.0, dtype=torch.bfloat16, device="cuda"),
                gH=torch.full((T + 2, 4, 4), 9.0, device="cuda"))
    head = {k: v[:T] for k, v in full.items()}
    ckpt = (head["codes"], head["scales"])
    gpu_lib.stream_mix_ckpt(x, H, out=head["out"], ckpt=ckpt)
    gpu_lib.stream_mix_bwd_ckpt(ckpt, H, g, out=(head["gx"], head["gH"]))
    for k, v in full.items():
        assert bool((v[T:] == (77 if v.dtype == torch.uint8 else 9.0)).all()), k


def test_projected_mix_gradients(gpu_lib):
    """The autograd form: against the formulas, and against central
    differences in float64 (at an x that its checkpoint holds exactly, so that
    the checkpointed gradient is the function's own)."""
    T, C = 33, 136
    x0 = rand((T, 4, C), 41)
    for fmt in FMTS:
        x = gpu_lib.ckpt_unpack(*gpu_lib.ckpt_pack(x0, format=fmt), format=fmt).requires_grad_(True)
        logits = torch.from_numpy(W.logits_batch("normal1", T, 42)).cuda().requires_grad_(True)
        g = rand((T, 4, C), 43)
        y = gpu_lib.projected_mix(x, logits, format=fmt)
        gx, gl = torch.autograd.grad(y, (x, logits), g)
        x64, l64, g64 = f64(x.detach()), logits.detach().cpu().numpy().astype(np.float64), f64(g)
        H = birkhoff_project(l64)
        gH = np.einsum("tic,tjc->tij", g64, x64)
        ref = birkhoff_project_bwd(H, gH)
        # the projection gradient's bar: 1e-4 of its largest entry + 1e-5 of dL/dH's
        bar = 1e-4 * np.abs(ref).max((1, 2), keepdims=True) + 1e-5 * np.abs(gH).max((1, 2), keepdims=True)
        assert (np.abs(gl.cpu().numpy() - ref) <= bar).all()
        refx = np.einsum("tij,tic->tjc", H, g64)
        magx = np.einsum("tij,tic->tjc", H, np.abs(g64))
        # H is within 1e-5 of the oracle's; then one bf16 rounding
        assert (np.abs(f64(gx) - refx) <= 2.0 ** -8 * np.abs(refx) + 1e-6 * magx
                + 1e-5 * np.abs(g64).sum(1, keepdims=True)).all()
        d = np.random.Generator(np.random.PCG64(44)).standard_normal((T, 4, 4))
        h = 1e-5
        loss = lambda l: np.einsum("tij,tij->t", birkhoff_project(l), gH)
        diff = (loss(l64 + h * d) - loss(l64 - h * d)) / (2 * h)
        along = (gl.cpu().numpy().astype(np.float64) * d).sum((1, 2))
        # differences: h^2 times third derivatives (each below 8 |gH| |d|^3) and rounding / h
        size = np.abs(gH).sum((1, 2))
        assert (np.abs(along - diff) <= bar[:, 0, 0] * np.abs(d).sum((1, 2)) + 1e-6 * size).all()


def _layer_case(T, C, seed, wscale=1.0):
    g = np.random.Generator(np.random.PCG64(seed))
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).cuda()
    D = 4 * C
    return (bf(g.standard_normal((T, 4, C)) * np.exp(g.standard_normal((1, 1, C)) / 2)),
            bf(g.standard_normal((24, D)) * wscale * 2.0 / np.sqrt(D)), bf(g.standard_normal((T, C))),
            bf(g.standard_normal((T, 4, C))), bf(g.standard_normal((T, C))))


def check_layer_fwd(gpu_lib, fw, x, Wt, f):
    """The forward beside the checkpoints: the read half's maps and u bit for
    bit, with many tokens all of layer_fwd's; x_out from those maps."""
    T = x.shape[0]
    read = gpu_lib.layer_read(x, Wt)
    for k in read:
        assert torch.equal(fw[k], read[k]), k
    if T > (8192 if x.shape[2] >= 2048 else 2048):
        fw0 = gpu_lib.layer_fwd(x, Wt, f)
        for k in fw0:
            assert torch.equal(fw[k], fw0[k]), k
    post, res = fw["H_post"].double()[:, :, None], fw["H_res"].double()
    ref = post * f.double()[:, None] + torch.matmul(res, x.double())
    mag = post * f.double().abs()[:, None] + torch.matmul(res, x.double().abs())
    assert bool(((fw["x_out"].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 5 * U * mag).all())


def check_layer_bwd(bw, fwd, xh, W64, fh, g64, u64):
    """The layer backward's outputs against the oracle for xhat, fhat and the
    kernel's own forward maps."""
    T, n, C = xh.shape
    ob = K.layer_bwd(xh, W64, fh, g64, u64, fwd)
    r, Hp, Ho, Hr, lg = (fwd[k] for k in ("rms", "H_pre", "H_post", "H_res", "logits"))
    dl = ob["dlogits"]

    def close(name, got, want, bound):
        err = np.abs(got - want)
        at = np.unravel_index(np.argmax(err - bound), err.shape)
        assert (err <= bound).all(), f"{name}: {err[at]:.3e} > {np.broadcast_to(bound, err.shape)[at]:.3e} at {at}"

    dH = np.concatenate([ob["d_pre"], ob["d_post"], ob["d_res"].reshape(T, 16)], axis=1)
    lbar = 1e-4 * np.abs(dl).max(1, keepdims=True) + 1e-5 * np.abs(dH).max(1, keepdims=True)
    close("grad_logits", bw["grad_logits"], dl, lbar)
    close("grad_f", bw["grad_f"], ob["df"],
          2.0 ** -8 * np.abs(ob["df"]) + 5 * U * np.einsum("ti,tic->tc", Ho, np.abs(g64)))
    S = (np.einsum("tij,tic->tjc", Hr, np.abs(g64)) + Hp[:, :, None] * np.abs(u64)[:, None, :]
         + (np.abs(dl) @ np.abs(W64)).reshape(T, n, C) / r[:, None, None]
         + np.abs(xh) * np.abs((dl * lg).sum(1) / (n * C) / r ** 2)[:, None, None])
    close("grad_x", bw["grad_x"], ob["dx"], 2.0 ** -8 * np.abs(ob["dx"]) + 2e-4 * S + 1e-6)
    # grad_W: from the kernel's own grad_logits the product is fp32-like: dl / r
    # in three bf16 parts (off by 2^-24 of it at most), 1/r and the product
    # rounded (3 u), and a sum of T terms in chains of MFMA steps whose
    # partial sums err by at most (T + 16) u of sum|terms|
    xn = xh.reshape(T, -1)
    gl = bw["grad_logits"] / r[:, None]
    close("grad_W", bw["grad_W"], gl.T @ xn, (T + 20) * U * (np.abs(gl).T @ np.abs(xn)) + 1e-30)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,C", [(1, 64), (37, 64), (64, 128), (130, 192), (300, 576), (2048, 256), (1, 7168), (5, 1088), (66, 2624), (70, 448),
                                 (2049, 576), (2100, 64), (2100, 2048)])
def test_layer_ckpt(gpu_lib, T, C, fmt):
    print(f"layer ckpt T={T} C={C} {fmt}", flush=True)
    x, Wt, f, g, du = _layer_case(T, C, T + C)
    fw, ck = gpu_lib.layer_fwd_ckpt(x, Wt, f, format=fmt)
    check_layer_fwd(gpu_lib, fw, x, Wt, f)
    for k, t in (("x", x), ("f", f)):
        c, s = gpu_lib.ckpt_pack(t, format=fmt)
        assert torch.equal(ck[k][0], c) and torch.equal(ck[k][1], s), k
    nan = {k: torch.full(sh, float("nan"), dtype=dt, device="cuda")
           for k, (sh, dt) in gpu_lib.ops._bwd_shapes(T, 4, C).items()}
    ws = torch.full((gpu_lib.layer_ckpt_workspace(T, C, x.device).numel(),), 0xFF, dtype=torch.uint8, device="cuda")
    bw = gpu_lib.layer_bwd_ckpt(ck, Wt, fw, g, du, format=fmt, out=nan, workspace=ws)
    xh, fh = (f64(gpu_lib.ckpt_unpack(*ck[k], format=fmt)) for k in ("x", "f"))
    dbl = lambda d: {k: f64(v) for k, v in d.items()}
    check_layer_bwd(dbl(bw), dbl(fw), xh, f64(Wt), fh, f64(g), f64(du))


def test_layer_ckpt_of_exact_values_is_the_layer_backward(gpu_lib):
    """Where x and f are held exactly, the backward is the plain layer's: the
    oracle's own layer backward, which knows nothing of checkpoints."""
    T, C = 96, 128
    x, Wt, f, g, du = _layer_case(T, C, 5)
    for fmt in FMTS:
        xe, fe = (gpu_lib.ckpt_unpack(*gpu_lib.ckpt_pack(t, format=fmt), format=fmt) for t in (x, f))
        fw, ck = gpu_lib.layer_fwd_ckpt(xe, Wt, fe, format=fmt)
        bw = gpu_lib.layer_bwd_ckpt(ck, Wt, fw, g, du, format=fmt)
        ref = gpu_lib.layer_bwd(xe, Wt, fe, fw, g, du)
        ob = o_layer_bwd(f64(xe), f64(Wt), f64(fe), f64(g), f64(du))
        dl = ob["dlogits"]
        assert (np.abs(f64(bw["grad_logits"]) - dl) <= 2e-4 * np.abs(dl).max()).all()
        assert np.abs(f64(bw["grad_W"]) - ob["dW"]).max() <= 2e-4 * (np.abs(dl).T @ np.abs(f64(xe).reshape(T, -1))).max()
        assert torch.equal(bw["grad_f"], ref["grad_f"])


def test_layer_ckpt_full_width(gpu_lib):
    """T = 8192 + 37, C = 7168: sampled tokens' grad_x and grad_f, every
    grad_logits and every grad_W entry, the reference in 64 bits on the GPU
    from the kernel's own maps, in pieces of tokens."""
    T, C = 8192 + 37, 7168
    inp = W.layer_inputs(T, C, seed=50)
    x, Wt, f, g, du = inp["x"], inp["W"], inp["f"], inp["dx_out"], inp["du"]
    fw, ck = gpu_lib.layer_fwd_ckpt(x, Wt, f, format="e4m3")
    bw = gpu_lib.layer_bwd_ckpt(ck, Wt, fw, g, du, format="e4m3")
    xh = gpu_lib.ckpt_unpack(*ck["x"], format="e4m3")
    gl = bw["grad_logits"].double() / fw["rms"].double()[:, None]
    ref = torch.zeros(24, 4 * C, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for t in range(0, T, 1024):
        xd = xh[t:t + 1024].view(-1, 4 * C).double()
        ref += gl[t:t + 1024].t() @ xd
        mag += gl[t:t + 1024].abs().t() @ xd.abs()
    # as in check_layer_bwd, in the random-walk form: 4 sqrt(T) u sum|terms|
    assert bool(((bw["grad_W"].double() - ref).abs() <= 4 * T ** 0.5 * U * mag).all())
    idx = torch.tensor([0, 1, 63, 64, 4000, T - 38, T - 2, T - 1], device="cuda")
    pick = lambda t: f64(t[idx])
    fwd = {k: pick(fw[k]) for k in ("rms", "logits", "H_pre", "H_post", "H_res")}
    sub = {k: pick(bw[k]) for k in ("grad_x", "grad_f", "grad_logits")}
    fh = gpu_lib.ckpt_unpack(*ck["f"], format="e4m3")
    own = {"grad_W": (sub["grad_logits"] / fwd["rms"][:, None]).T @ pick(xh).reshape(8, -1)}
    check_layer_bwd({**sub, **own}, fwd, pick(xh), f64(Wt), pick(fh), pick(g), pick(du))


def test_empty_layer_and_tensors(gpu_lib):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    c, s = gpu_lib.ckpt_pack(z(0, 64))
    assert c.shape == (0, 64) and s.shape == (0, 2)
    assert gpu_lib.ckpt_unpack(c, s).shape == (0, 64)
    fw, ck = gpu_lib.layer_fwd_ckpt(z(0, 4, 64), rand((24, 256), 1), z(0, 64))
    bw = gpu_lib.layer_bwd_ckpt(ck, rand((24, 256), 1), fw, z(0, 4, 64), z(0, 64))
    assert bool((bw["grad_W"] == 0).all())


def test_graph_replays_and_streams(gpu_lib):
    """A whole training step of the mix and the layer captured once and
    replayed with eager work between, and the same on a side stream."""
    T, C = 130, 192
    x, Wt, f, g, du = _layer_case(T, C, 9)
    H = gpu_lib.birkhoff_fwd(rand((T, 4, 4), 10, torch.float32))
    ws = gpu_lib.layer_ckpt_workspace(T, C, x.device)

    def step():
        out, ck = gpu_lib.stream_mix_ckpt(x, H, format="int8")
        gx, gH = gpu_lib.stream_mix_bwd_ckpt(ck, H, g, format="int8")
        fw, lk = gpu_lib.layer_fwd_ckpt(x, Wt, f)
        bw = gpu_lib.layer_bwd_ckpt(lk, Wt, fw, g, du, workspace=ws)
        q = gpu_lib.mx4_dequantize(*gpu_lib.mx4_quantize(x.view(-1, C)))
        return [out, gx, gH, *bw.values(), fw["x_out"], q]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(4):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep
        step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refuses_short_buffers(gpu_lib):
    T, C = 16, 64
    x, Wt, f, g, du = _layer_case(T, C, 11)
    H = rand((T, 4, 4), 12, torch.float32)
    codes = torch.full((T, 4, C), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((T, 4, 2), 77, dtype=torch.uint8, device="cuda")
    bad = [lambda: gpu_lib.ckpt_pack(x, out=(codes[:-1], scales)),
           lambda: gpu_lib.ckpt_pack(x, out=(codes, scales[..., :1].contiguous())),
           lambda: gpu_lib.ckpt_pack(x.transpose(0, 1)),
           lambda: gpu_lib.ckpt_unpack(codes, scales[:-1]),
           lambda: gpu_lib.ckpt_unpack(codes, scales, out=x[:-1]),
           lambda: gpu_lib.stream_mix_ckpt(x, H, ckpt=(codes, scales[:-1])),
           lambda: gpu_lib.stream_mix_ckpt(x, H, logits=H),
           lambda: gpu_lib.stream_mix_ckpt(x, H[:-1]),
           lambda: gpu_lib.stream_mix_bwd_ckpt((codes[:-1], scales), H, g),
           lambda: gpu_lib.stream_mix_bwd_ckpt((codes, scales), H[:-1], g),
           lambda: gpu_lib.layer_fwd_ckpt(x, Wt, f, ckpt=dict(x=(codes, scales), f=(codes, scales))),
           lambda: gpu_lib.mx4_dequantize(codes.view(-1, C), scales.view(-1, 2))]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", k)
    with pytest.raises(TypeError):
        gpu_lib.stream_mix_bwd_ckpt((codes.float(), scales), H, g)
    with pytest.raises(gpu_lib.MHCError):
        gpu_lib.ckpt_pack(torch.zeros(4, 12, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert bool((codes == 77).all()) and bool((scales == 77).all())
