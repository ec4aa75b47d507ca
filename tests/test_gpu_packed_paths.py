"""The checkpoint and 4-bit kernels on every path that their sizes choose:
each tile, scale copy and epilogue of the products with several stages,
several panels of the few-row kernel, the loops over many tokens, offsets past
32 bits, and blocks that are not finite.

Bars are those of test_gpu_mx4.py and test_gpu_ckpt.py, derived there, except
  grad_H      a lane of a kernel of W lanes to a token adds 8 ceil(C / 8W)
              exact products in a chain, then come the levels of the sum over
              the lanes (4, 6 and 6 + 2 for W = 16, 64 and 256), so |d| <=
              (8 ceil(C / 8W) + levels) u sum|terms|
"""
import numpy as np
import pytest
import torch

import test_gpu_ckpt as ck_tests
import workloads as W
from test_gpu_ckpt import FMTS, U, _layer_case, f64, rand
from test_gpu_mx4 import HALF, close, operand, values

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def route(M, N, K):
    """(kernel, scale copies, more than one stage or panel): the choice in
    csrc/mx4.hip, written again."""
    cdiv = lambda a, b: -(-a // b)
    if M <= 16 or cdiv(M, 16) * cdiv(N, 16) <= 512:
        rows = next(r for r in (1, 2, 4, 8, 16) if r >= min(M, 16))
        panels = cdiv(cdiv(K, 256), 70 * 1024 // ((16 + rows) * 136))
        return "few", "words" if K % 128 == 0 else "bytes", panels > 1
    t256, t128 = cdiv(M, 256) * cdiv(N, 256), cdiv(M, 128) * cdiv(N, 128)
    tile = "256" if t256 >= 192 else ("128x2" if t128 > 256 else ("128x3" if t128 > 128 else "64"))
    return tile, "pairs" if K % 512 == 0 else ("words" if K % 256 == 0 else "tail"), K > 256


PRODUCTS = [(130, 1032, 1024), (130, 1032, 768), (130, 1032, 800), (1200, 2056, 1024), (1200, 2056, 768),
            (1200, 2056, 800), (2100, 2304, 1024), (2100, 2304, 768), (2100, 2304, 800), (3600, 3400, 1024),
            (3600, 3400, 768), (3600, 3400, 800), (9, 136, 1152), (9, 136, 800), (1, 72, 8192), (5, 264, 8224),
            (16, 72, 4480), (40, 264, 5120), (50, 264, 5152)]


def test_products_cover_every_route():
    want = {(t, m, True) for t in ("256", "128x2", "128x3", "64") for m in ("pairs", "words", "tail")}
    want |= {("few", m, p) for m in ("words", "bytes") for p in (False, True)}
    assert {route(*s) for s in PRODUCTS} == want


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_and_write_back(gpu_lib, M, N, K):
    print(f"paths {M}x{N}x{K} {route(M, N, K)}", flush=True)
    a, b = operand(M, K, M + K), operand(N, K, N + K + 1)
    va, vb = values(a), values(b)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((M + 2, N), 3.0, dtype=dt, device="cuda")
        y = gpu_lib.mx4_matmul(a, b, out_dtype=dt, out=buf[:M])
        close(y, va, vb, dt, f"{dt}")
        assert bool((buf[M:] == 3.0).all())
    F, mF = va @ vb.t(), va.abs() @ vb.abs().t()
    x = rand((M, 4, N), 7)
    post, res = torch.rand(M, 4, device="cuda"), torch.softmax(rand((M, 4, 4), 8, torch.float32), -1)
    buf = torch.full((M + 1, 4, N), 5.0, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    out = gpu_lib.mx4_write_back(a, b, x, post, res, out=buf[:M], f_out=f)
    assert torch.equal(f, gpu_lib.mx4_matmul(a, b)) and bool((buf[M:] == 5.0).all())
    for i in range(4):  # a stream at a time: the reference is large
        pd, rd = post[:, i, None].double(), res[:, i, None].double()
        mix = torch.matmul(rd, x.double())[:, 0]
        ref = pd * F + mix
        mag = pd * F.abs() + torch.matmul(rd, x.double().abs())[:, 0]
        bound = pd * ((K / 32 + 40) * U * mF) + 5 * U * mag + 2.0 ** -8 * ref.abs()
        assert bool(((out[:, i].double() - ref).abs() <= bound).all()), i


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_nan_scales_stay_in_their_rows(gpu_lib, M, N, K):
    print(f"nan {M}x{N}x{K} {route(M, N, K)}", flush=True)
    a, b = operand(M, K, 1), operand(N, K, 2)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    for m, k in ((0, 0), (M // 2, K // 32 - 1), (M - 1, K // 64)):
        a[1][m, k] = 255
        want[m] = True
    for n, k in ((5, K // 32 - 1), (N - 1, 0)):
        b[1][n, k] = 255
        want[:, n] = True
    assert torch.equal(torch.isnan(gpu_lib.mx4_matmul(a, b, out_dtype=torch.float32)), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 64, 8192), (4, 136, 8192), (1, 64, 32768), (3, 200, 10912), (2, 72, 16384)])
def test_quantising_product_of_several_panels(gpu_lib, M, N, K, dtype):
    """Few rows whose values the product quantises itself, K in two to five
    panels: against the packed operand and bit for bit from call to call."""
    assert M * K <= 32768 and route(M, N, K)[2]
    print(f"values {M}x{N}x{K} {dtype}", flush=True)
    x = rand((M, K), M + N, dtype) * torch.exp(rand((1, K), 5, torch.float32)).to(dtype)
    b = operand(N, K, K)
    y = gpu_lib.mx4_matmul(x, b, out_dtype=dtype)
    close(y, values(gpu_lib.mx4_quantize(x)), values(b), dtype)
    assert all(torch.equal(y, gpu_lib.mx4_matmul(x, b, out_dtype=dtype)) for _ in range(5))


def test_sublayer_of_many_tokens_is_its_own_maps_and_codes(gpu_lib):
    """16384 tokens of 4096: ten calls agree bit for bit, u4 is the quantised
    bf16 u, and x_out is the combination of exactly these."""
    T, C = 16384, 4096
    x, Wt = rand((T, 4, C), 1), rand((24, 4 * C), 2, scale=2.0 / (4 * C) ** 0.5)
    w = gpu_lib.mx4_quantize(rand((C, C), 3, scale=C ** -0.5))
    r = gpu_lib.layer_read(x, Wt, mx4=True, keep_u=True)
    out = gpu_lib.mx4_write_back(r["u"], w, x, r["H_post"], r["H_res"])
    for p, q in zip(r["u"], gpu_lib.mx4_quantize(r["u_values"])):
        assert torch.equal(p, q)
    for _ in range(9):
        again = gpu_lib.layer_read(x, Wt, mx4=True)
        assert all(torch.equal(again[k], r[k]) for k in ("rms", "logits", "H_pre", "H_post", "H_res"))
        assert all(torch.equal(p, q) for p, q in zip(again["u"], r["u"]))
        assert torch.equal(out, gpu_lib.mx4_write_back(again["u"], w, x, again["H_post"], again["H_res"]))
    vb = gpu_lib.mx4_dequantize(*w, dtype=torch.float32).double()  # exact in fp32
    for t in range(0, T, 2048):
        s = slice(t, t + 2048)
        va = gpu_lib.mx4_dequantize(*(p[s].contiguous() for p in r["u"]), dtype=torch.float32).double()
        F, mF = va @ vb.t(), va.abs() @ vb.abs().t()
        for i in range(4):
            pd, rd = r["H_post"][s, i, None].double(), r["H_res"][s, i, None].double()
            ref = pd * F + torch.matmul(rd, x[s].double())[:, 0]
            mag = pd * F.abs() + torch.matmul(rd, x[s].double().abs())[:, 0]
            bound = pd * ((C / 32 + 40) * U * mF) + 5 * U * mag + 2.0 ** -8 * ref.abs()
            assert bool(((out[s, i].double() - ref).abs() <= bound).all()), (t, i)


# ---------------------------------------------------------------------------
# mix and layer
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,C", [(241, 72), (300, 200), (33000, 16), (40000, 136), (8200, 264), (16400, 520), (9, 512),
                                 (2049, 520), (3, 5792), (100, 520)])
def test_mix_backward_of_every_width(gpu_lib, T, C, fmt):
    """16, 64 and 256 lanes to a token, and more tokens than the grid takes at
    once."""
    print(f"mix T={T} C={C} {fmt}", flush=True)
    x, g = rand((T, 4, C), T + C), rand((T, 4, C), T + C + 1)
    H = gpu_lib.birkhoff_fwd(rand((T, 4, 4), 3, torch.float32))
    out, ckpt = gpu_lib.stream_mix_ckpt(x, H, format=fmt)
    assert torch.equal(out, gpu_lib.stream_mix(x, H))
    assert all(torch.equal(p, q) for p, q in zip(ckpt, gpu_lib.ckpt_pack(x, format=fmt)))
    gx, gH = gpu_lib.stream_mix_bwd_ckpt(ckpt, H, g, format=fmt)
    assert torch.equal(gx, gpu_lib.stream_mix_bwd(x, H, g)[0])
    xt = gpu_lib.ckpt_unpack(*ckpt, format=fmt).double().transpose(1, 2).contiguous()
    ref, mag = torch.matmul(g.double(), xt), torch.matmul(g.double().abs(), xt.abs())
    lanes, levels = (16, 4) if C <= 256 else ((256, 8) if T <= 2048 and C > 512 else (64, 6))
    assert bool(((gH.double() - ref).abs() <= (8 * -(-C // (8 * lanes)) + levels) * U * mag).all())


def layer_step(gpu_lib, T, C, fmt, seed):
    x, Wt, f, g, du = _layer_case(T, C, seed)
    fw, ck = gpu_lib.layer_fwd_ckpt(x, Wt, f, format=fmt)
    return (x, Wt, f, g, du), fw, ck, gpu_lib.layer_bwd_ckpt(ck, Wt, fw, g, du, format=fmt)


@pytest.mark.parametrize("T,C,fmt", [(9000, 64, "int8"), (16400, 64, "e4m3"), (33000, 64, "int8"), (16400, 128, "e4m3"),
                                     (9000, 320, "e4m3"), (16400, 320, "int8")])
def test_layer_of_many_tokens(gpu_lib, T, C, fmt):
    """8 and 16 tokens to a wave in the pass over the dots, narrow and wide."""
    print(f"layer T={T} C={C} {fmt}", flush=True)
    (x, Wt, f, g, du), fw, ck, bw = layer_step(gpu_lib, T, C, fmt, T + C)
    ck_tests.check_layer_fwd(gpu_lib, fw, x, Wt, f)
    xh, fh = (f64(gpu_lib.ckpt_unpack(*ck[k], format=fmt)) for k in ("x", "f"))
    dbl = lambda d: {k: f64(v) for k, v in d.items()}
    ck_tests.check_layer_bwd(dbl(bw), dbl(fw), xh, f64(Wt), fh, f64(g), f64(du))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,C", [(1, 64), (37, 192), (300, 576), (2100, 2048), (2049, 64)])
def test_layer_forward_with_sinkhorn(gpu_lib, T, C, fmt):
    print(f"layer sinkhorn T={T} C={C} {fmt}", flush=True)
    x, Wt, f, _, _ = _layer_case(T, C, T + C)
    fw, ck = gpu_lib.layer_fwd_ckpt(x, Wt, f, format=fmt, solver="sinkhorn")
    read = gpu_lib.layer_read(x, Wt, solver="sinkhorn")
    assert all(torch.equal(fw[k], read[k]) for k in read)
    for k, t in (("x", x), ("f", f)):
        assert all(torch.equal(p, q) for p, q in zip(ck[k], gpu_lib.ckpt_pack(t, format=fmt)))
    post, res = fw["H_post"].double()[:, :, None], fw["H_res"].double()
    ref = post * f.double()[:, None] + torch.matmul(res, x.double())
    mag = post * f.double().abs()[:, None] + torch.matmul(res, x.double().abs())
    assert bool(((fw["x_out"].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 5 * U * mag).all())


@pytest.mark.parametrize("T,C", [(5, 64), (70, 576), (2100, 128), (2100, 320)])
def test_projection_gradient_without_the_ridge(gpu_lib, T, C):
    """grad_logits of H_res = 1/4 throughout and dL/dH_res = G with equal rows
    (-a, -a, -a, a): zero, as every G is whose rows are equal.

    The solve's unknown is -2a three times.  Its reduced Laplacian is I - J/4
    with the eigenvalue 1/4 there, and the ridge, 8 eps times its trace 2.25,
    is 2.1e-6: one solve leaves 8.6e-6 of 2a, which is 3.2e-6 a in the
    gradient.  After the second only the rounding of -2a is left, at most 2 u a
    in each unknown: the differences behind it are between nearly equal numbers
    and exact.  A gradient is 1/4 of the sum of 3 such differences a quarter
    each, two of them of at most 4 u a and one of 2 u a: at most 0.63 u a."""
    s = 1.0 + torch.arange(T, device="cuda") % 15  # whole numbers that e4m3 and int8 hold
    sign = torch.tensor([-1.0, -1.0, -1.0, 1.0], device="cuda")
    x = (s[:, None, None] * sign[None, :, None]).expand(T, 4, C).bfloat16().contiguous()
    zeros = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    ones = torch.ones(T, 4, C, dtype=torch.bfloat16, device="cuda")
    Wt = torch.zeros(24, 4 * C, dtype=torch.bfloat16, device="cuda")
    fwd = dict(rms=torch.ones(T, device="cuda"), logits=torch.zeros(T, 24, device="cuda"),
               H_pre=torch.full((T, 4), 0.5, device="cuda"), H_post=torch.full((T, 4), 0.5, device="cuda"),
               H_res=torch.full((T, 4, 4), 0.25, device="cuda"))
    for fmt in FMTS:
        ck = dict(x=gpu_lib.ckpt_pack(x, format=fmt), f=gpu_lib.ckpt_pack(zeros, format=fmt))
        assert torch.equal(gpu_lib.ckpt_unpack(*ck["x"], format=fmt), x)
        gl = gpu_lib.layer_bwd_ckpt(ck, Wt, fwd, ones, zeros, format=fmt)["grad_logits"]
        assert not bool(gl[:, :8].any())
        assert bool((gl[:, 8:].abs() <= U * (C * s)[:, None]).all()), float((gl.abs() / (C * s)[:, None]).max()) / U


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------

def same(a, b):
    """Equal values, NaN in the same places."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,C", [(9, 72), (40, 264), (60, 1000)])
def test_mix_of_non_finite_blocks(gpu_lib, T, C, fmt):
    x, g = rand((T, 4, C), 1), rand((T, 4, C), 2)
    H = gpu_lib.birkhoff_fwd(rand((T, 4, 4), 3, torch.float32))
    _, clean = gpu_lib.stream_mix_ckpt(x, H, format=fmt)
    gx0, gH0 = gpu_lib.stream_mix_bwd_ckpt(clean, H, g, format=fmt)
    bad = torch.zeros(T, 4, dtype=torch.bool, device="cuda")
    for t, j, c, v in ((0, 1, 0, float("nan")), (3, 3, C - 1, float("inf")), (T - 1, 0, C // 2, float("-inf"))):
        x[t, j, c] = v
        bad[t, j] = True
    out, ckpt = gpu_lib.stream_mix_ckpt(x, H, format=fmt)
    assert same(out, gpu_lib.stream_mix(x, H))
    assert all(torch.equal(p, q) for p, q in zip(ckpt, gpu_lib.ckpt_pack(x, format=fmt)))
    gx, gH = gpu_lib.stream_mix_bwd_ckpt(ckpt, H, g, format=fmt)
    assert torch.equal(gx, gx0)
    assert torch.equal(torch.isnan(gH), bad[:, None, :].expand(T, 4, 4))
    assert torch.equal(gH[~torch.isnan(gH)], gH0[~torch.isnan(gH)])
    x.zero_()  # and nothing but zeros
    out, ckpt = gpu_lib.stream_mix_ckpt(x, H, format=fmt)
    assert not bool(out.any()) and not bool(gpu_lib.stream_mix_bwd_ckpt(ckpt, H, g, format=fmt)[1].any())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,C", [(7, 64), (70, 576), (2100, 128), (2050, 320)])
def test_layer_of_non_finite_tokens(gpu_lib, T, C, fmt):
    """A token whose x holds an infinity or a NaN spoils itself and grad_W; one
    whose f does, only what comes from f."""
    x, Wt, f, g, du = _layer_case(T, C, 3)
    fw0, ck0 = gpu_lib.layer_fwd_ckpt(x, Wt, f, format=fmt)
    bw0 = gpu_lib.layer_bwd_ckpt(ck0, Wt, fw0, g, du, format=fmt)
    names = ("rms", "logits", "H_pre", "H_post", "H_res", "u", "x_out")

    f2 = f.clone()
    f2[2, 5] = float("inf")
    fw, ck = gpu_lib.layer_fwd_ckpt(x, Wt, f2, format=fmt)
    assert all(torch.equal(fw[k], fw0[k]) for k in names[:-1])
    bw = gpu_lib.layer_bwd_ckpt(ck, Wt, fw, g, du, format=fmt)
    assert torch.equal(bw["grad_f"], bw0["grad_f"])
    others = torch.arange(T, device="cuda") != 2
    for k in ("grad_x", "grad_logits"):
        assert torch.equal(bw[k][others], bw0[k][others]), k
    from_f = torch.arange(24, device="cuda").view(24, 1).expand(24, 4 * C) // 4 == 1
    assert torch.equal(torch.isnan(bw["grad_logits"][2]), from_f[:, 0])
    assert torch.equal(torch.isnan(bw["grad_W"]), from_f)
    assert torch.equal(bw["grad_W"][~from_f], bw0["grad_W"][~from_f])
    assert bool(torch.isnan(bw["grad_x"][2]).all())

    for v in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[2, 1, C - 1] = v
        fw, ck = gpu_lib.layer_fwd_ckpt(x2, Wt, f, format=fmt)
        read = gpu_lib.layer_read(x2, Wt)
        for k in names:
            assert torch.equal(fw[k][others], fw0[k][others]), k
            if k in read:
                assert same(fw[k], read[k]), k
        bw = gpu_lib.layer_bwd_ckpt(ck, Wt, fw, g, du, format=fmt)
        for k in ("grad_x", "grad_f", "grad_logits"):
            assert torch.equal(bw[k][others], bw0[k][others]), k
        assert bool(torch.isnan(bw["grad_logits"][2]).any()) and bool(torch.isnan(bw["grad_x"][2]).any())
        assert bool(torch.isnan(bw["grad_W"]).any())


def test_read_of_zero_and_non_finite_tokens(gpu_lib):
    for T, C in ((40, 576), (2100, 128)):
        x, Wt = rand((T, 4, C), 1), rand((24, 4 * C), 2, scale=2.0 / (4 * C) ** 0.5)
        r0 = gpu_lib.layer_read(x, Wt, mx4=True, keep_u=True)
        x[1], x[3, 2, 7] = 0.0, float("nan")
        r = gpu_lib.layer_read(x, Wt, mx4=True, keep_u=True)
        others = torch.ones(T, dtype=torch.bool, device="cuda")
        others[1] = others[3] = False
        for k in ("rms", "logits", "H_pre", "H_post", "H_res", "u_values"):
            assert torch.equal(r[k][others], r0[k][others]), k
        assert all(torch.equal(p[others], q[others]) for p, q in zip(r["u"], r0["u"]))
        assert not bool(r["logits"][1].any()) and not bool(r["u_values"][1].any())
        assert bool(((r["H_pre"][1] - 0.5).abs() <= 1e-6).all()) and bool(((r["H_res"][1] - 0.25).abs() <= 1e-5).all())
        assert bool((r["u"][1][3] == 255).all()) and bool((r["u"][1][1] == 2).all())  # scale bytes: NaN, the least


def test_linear_of_non_finite_rows(gpu_lib):
    """An infinity in x makes its row of y NaN and, through the quantised
    transpose, its block of 32 columns of grad_w; grad_x is unchanged."""
    M, N, K = 96, 160, 128
    x, w, gy = rand((M, K), 1), rand((N, K), 2), rand((M, N), 3)

    def step():
        leaves = [t.clone().requires_grad_(True) for t in (x, w)]
        y = gpu_lib.mx4_linear(*leaves)
        return [y.detach(), *torch.autograd.grad(y, leaves, gy)]

    y0, gx0, gw0 = step()
    x[7, 40] = float("inf")
    y, gx, gw = step()
    rows = torch.arange(M, device="cuda") == 7
    cols = torch.arange(K, device="cuda") // 32 == 1
    assert torch.equal(torch.isnan(y), rows[:, None].expand(M, N)) and torch.equal(y[~rows], y0[~rows])
    assert torch.equal(gx, gx0)
    assert torch.equal(torch.isnan(gw), cols[None].expand(N, K)) and torch.equal(gw[:, ~cols], gw0[:, ~cols])


# ---------------------------------------------------------------------------
# offsets past 32 bits: the last rows come out as the same rows alone
# ---------------------------------------------------------------------------

def test_mix_past_32_bit_offsets(gpu_lib):
    T, C, n = (1 << 32) // (4 * 4096) + 40, 4096, 64
    x, g = (torch.zeros((T, 4, C), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-n:], g[-n:] = rand((n, 4, C), 1), rand((n, 4, C), 2)
    H = torch.full((T, 4, 4), 0.25, device="cuda")
    H[-n:] = gpu_lib.birkhoff_fwd(rand((n, 4, 4), 3, torch.float32))
    out, ckpt = gpu_lib.stream_mix_ckpt(x, H, format="int8")
    tail = [t[-n:].contiguous() for t in (x, g, H)]
    out1, ckpt1 = gpu_lib.stream_mix_ckpt(tail[0], tail[2], format="int8")
    assert torch.equal(out[-n:], out1) and not bool(out[:-n].any())
    assert all(torch.equal(p[-n:], q) for p, q in zip(ckpt, ckpt1)) and not bool(ckpt[0][:-n].any())
    del out, x
    gx, gH = gpu_lib.stream_mix_bwd_ckpt(ckpt, H, g, format="int8")
    xt = gpu_lib.ckpt_unpack(*ckpt1, format="int8").double().transpose(1, 2).contiguous()
    ref, mag = torch.matmul(tail[1].double(), xt), torch.matmul(tail[1].double().abs(), xt.abs())
    bound = (8 * C // 512 + 6) * U * mag  # 64 lanes to a token
    assert bool(((gH[-n:].double() - ref).abs() <= bound).all()) and not bool(gH[:-n].any())
    assert torch.equal(gx[-n:], gpu_lib.stream_mix_bwd(tail[0], tail[2], tail[1])[0]) and not bool(gx[:-n].any())


def test_layer_past_32_bit_offsets(gpu_lib):
    """Tokens in front are zeros, the last 8256 are not: per token everything
    is what these alone give, and grad_W is their sum."""
    C, n = 7168, 8256
    T = (1 << 32) // (4 * C) // 64 * 64 + 64 + n
    x1, Wt, f1, g1, du1 = _layer_case(n, C, 5)
    whole = []
    for t in (x1, f1, g1, du1):
        z = torch.zeros((T, *t.shape[1:]), dtype=t.dtype, device="cuda")
        z[-n:] = t
        whole.append(z)
    x, f, g, du = whole
    fw, ck = gpu_lib.layer_fwd_ckpt(x, Wt, f, format="e4m3")
    fw1, ck1 = gpu_lib.layer_fwd_ckpt(x1, Wt, f1, format="e4m3")
    assert all(torch.equal(fw[k][-n:], fw1[k]) for k in fw)
    assert all(torch.equal(p[-n:], q) for k in "xf" for p, q in zip(ck[k], ck1[k]))
    read = gpu_lib.layer_read(x, Wt)
    assert all(torch.equal(read[k][-n:], fw1[k]) for k in read)
    del read, x, f
    bw = gpu_lib.layer_bwd_ckpt(ck, Wt, fw, g, du, format="e4m3")
    bw1 = gpu_lib.layer_bwd_ckpt(ck1, Wt, fw1, g1, du1, format="e4m3")
    for k in ("grad_x", "grad_f", "grad_logits"):
        assert torch.equal(bw[k][-n:], bw1[k]) and not bool(bw[k][:-n].any()), k
    xh = gpu_lib.ckpt_unpack(*ck1["x"], format="e4m3").view(n, -1)
    gl = bw1["grad_logits"].double() / fw1["rms"].double()[:, None]
    ref = torch.zeros(24, 4 * C, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for t in range(0, n, 1032):
        xd = xh[t:t + 1032].double()
        ref += gl[t:t + 1032].t() @ xd
        mag += gl[t:t + 1032].abs().t() @ xd.abs()
    # zeros add nothing: the random-walk bar of n terms
    assert bool(((bw["grad_W"].double() - ref).abs() <= 4 * n ** 0.5 * U * mag).all())


def test_quantisers_past_32_bit_offsets(gpu_lib):
    C, n = 4096, 64
    R = (1 << 32) // C + 256
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    x[-n:] = tail = rand((n, C), 4)
    rows, cols = gpu_lib.mx4_quantize_both(x)
    r1, c1 = gpu_lib.mx4_quantize_both(tail)

    def ends(q, q1, along):
        for p, s in zip(q, q1):
            cut = p[-s.shape[0]:] if along == 0 else p[:, -s.shape[1]:]
            assert torch.equal(cut, s)

    ends(rows, r1, 0)
    ends(cols, c1, 1)
    assert not bool(rows[0][:-n].any()) and not bool(cols[0][:, :-n // 2].any())
    only = gpu_lib.mx4_quantize(x, transpose=True)
    assert all(torch.equal(p, q) for p, q in zip(only, cols))
    del only, cols
    q, ck = gpu_lib.mx4_quantize_ckpt(x, format="int8")
    assert all(torch.equal(a, b) for a, b in zip(q, rows))
    ends(ck, gpu_lib.ckpt_pack(tail, format="int8"), 0)
    del q, x
    back = gpu_lib.mx4_dequantize(*rows)
    assert torch.equal(back[-n:], gpu_lib.mx4_dequantize(*r1))
    del back, rows
    again = gpu_lib.mx4_requantize(*ck, format="int8")
    ends(again, gpu_lib.mx4_requantize(*gpu_lib.ckpt_pack(tail, format="int8"), format="int8"), 1)


@pytest.mark.parametrize("M,N,K", [(70000, 32768, 32),          # out past 2^31 elements, 256 x 256 tiles
                                   ((1 << 21) + 300, 8, 4096),  # a past 2^32 bytes
                                   (3, (1 << 21) + 40, 4128)])  # b past 2^32 bytes, few rows
def test_products_past_32_bit_offsets(gpu_lib, M, N, K):
    """Codes are zeros but in the last rows; every scale is 1."""
    print(f"large {M}x{N}x{K}", flush=True)
    ops, tails = [], []
    for rows, seed in ((M, 1), (N, 2)):
        codes = torch.zeros((rows, K // 2), dtype=torch.uint8, device="cuda")
        scales = torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda")
        n = min(rows, 64)
        c, s = operand(n, K, seed)
        codes[-n:], scales[-n:] = c, s
        ops.append((codes, scales))
        tails.append((c, s))
    y = gpu_lib.mx4_matmul(*ops)
    va, vb = (values(t) for t in tails)
    close(y[-va.shape[0]:, -vb.shape[0]:], va, vb, torch.bfloat16)
    assert not bool(y[:-64].any()) and not bool(y[:, :-64].any())


def test_write_back_past_32_bit_offsets(gpu_lib):
    T, C, K, n = (1 << 32) // (4 * 4096) + 300, 4096, 32, 300
    a = (torch.zeros((T, K // 2), dtype=torch.uint8, device="cuda"),
         torch.full((T, 1), 127, dtype=torch.uint8, device="cuda"))
    a1 = operand(n, K, 1)
    a[0][-n:], a[1][-n:] = a1
    b = operand(C, K, 2)
    x = torch.zeros((T, 4, C), dtype=torch.bfloat16, device="cuda")
    x[-n:] = x1 = rand((n, 4, C), 3)
    post, res = torch.rand(T, 4, device="cuda"), torch.softmax(rand((T, 4, 4), 8, torch.float32), -1)
    f = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    out = gpu_lib.mx4_write_back(a, b, x, post, res, f_out=f)
    F = values(a1) @ values(b).t()
    mF = values(a1).abs() @ values(b).abs().t()
    close(f[-n:], values(a1), values(b), torch.bfloat16)
    pd, rd = post[-n:].double()[:, :, None], res[-n:].double()
    ref = pd * F[:, None] + torch.matmul(rd, x1.double())
    mag = pd * F.abs()[:, None] + torch.matmul(rd, x1.double().abs())
    bound = pd * ((K / 32 + 40) * U * mF)[:, None] + 5 * U * mag + 2.0 ** -8 * ref.abs()
    assert bool(((out[-n:].double() - ref).abs() <= bound).all())
    assert not bool(out[:-n].any()) and not bool(f[:-n].any())


# ---------------------------------------------------------------------------
# two calls at once
# ---------------------------------------------------------------------------

def test_two_streams_at_once(gpu_lib):
    """Calls with workspaces (the maps' sums, the quantised operand, the layer
    backward) under way on two streams together."""
    T, C = 300, 576
    cases = [_layer_case(T, C, 60 + k) for k in range(2)]
    w = gpu_lib.mx4_quantize(rand((C, C), 61, scale=C ** -0.5))

    def step(case):
        x, Wt, f, g, du = case
        y = gpu_lib.mx4_matmul(f, w)
        fw, ck = gpu_lib.layer_fwd_ckpt(x, Wt, y)
        bw = gpu_lib.layer_bwd_ckpt(ck, Wt, fw, g, du)
        return [y, fw["x_out"], *bw.values()]

    want = [[t.clone() for t in step(c)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [[], []]
        for _ in range(4):
            for k, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[k].append(step(cases[k]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for k in range(2) for run in got[k] for a, b in zip(run, want[k]))
