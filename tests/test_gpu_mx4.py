"""GPU parity of the 4-bit products, the write-back product and the layer's
read half against float64.

Bar of a product: the terms are exact, the sum is fp32.  Within one matrix
instruction and along the chain of K / 64 of them (plus the joins of a split
sum) every addition errs by at most u = 2^-24 of a partial sum of |terms|, so
|d| <= (K / 32 + 40) u sum|terms|, then one rounding of the output: 2^-8 of it
in bf16, u in fp32.
"""
import numpy as np
import pytest
import torch

from oracle import birkhoff_project, packed as K_

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def rand(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def operand(R, C, seed, device="cuda"):
    """Random codes and scale bytes of a [R, C] MXFP4 matrix."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (R, C // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(120, 135, (R, C // 32), generator=g, dtype=torch.uint8)
    return codes.to(device), scales.to(device)


def values(q):
    """float64 values on the GPU of a (codes, scales) pair."""
    return torch.from_numpy(K_.values4(q[0].cpu().numpy(), q[1].cpu().numpy())).cuda()


def close(y, a, b, dtype, label=""):
    ref = a @ b.t()
    mag = a.abs() @ b.abs().t()
    bound = (a.shape[1] / 32 + 40) * U * mag + HALF[dtype] * ref.abs()
    err = (y.double() - ref).abs()
    assert bool((err <= bound).all()), f"{label}: {float((err - bound).max()):.3e} over at {int((err - bound).argmax())}"


SHAPES = [(1, 8, 32), (1, 7168, 4096), (3, 40, 96), (16, 136, 2080), (17, 64, 64), (33, 72, 512), (64, 200, 1056),
          (65, 8, 32), (100, 136, 160), (128, 128, 256), (130, 264, 288), (257, 1000, 480), (640, 4104, 96),
          (2100, 2056, 544), (4352, 4352, 256), (4100, 4360, 800),
          (130, 1032, 1056), (200, 1000, 512), (40, 2056, 96), (250, 496, 3200),
          (300, 1032, 2560), (300, 1032, 1280), (1200, 2056, 1024), (1200, 2056, 768), (2100, 2304, 1536),
          (4352, 4352, 1536), (4352, 4360, 768)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_packed(gpu_lib, M, N, K):
    print(f"mx4 matmul {M}x{N}x{K}", flush=True)
    a, b = operand(M, K, M + K), operand(N, K, N + K + 1)
    va, vb = values(a), values(b)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((M + 2, N), 3.0, dtype=dt, device="cuda")
        y = gpu_lib.mx4_matmul(a, b, out_dtype=dt, out=buf[:M])
        close(y, va, vb, dt, f"{M}x{N}x{K} {dt}")
        assert bool((buf[M:] == 3.0).all())
        assert torch.equal(y, gpu_lib.mx4_matmul(a, b, out_dtype=dt))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 7168, 7168), (2, 136, 1056), (16, 264, 5120), (11, 64, 96),
                                   (16, 64, 6144), (17, 200, 320), (300, 136, 288), (1, 64, 90144)])
def test_matmul_of_values(gpu_lib, M, N, K, dtype):
    print(f"mx4 matmul of values {M}x{N}x{K} {dtype}", flush=True)
    x = rand((M, K), M + N, dtype) * torch.exp(rand((1, K), 5, torch.float32)).to(dtype)
    b = operand(N, K, K)
    y = gpu_lib.mx4_matmul(x, b, out_dtype=dtype)
    qa = gpu_lib.mx4_quantize(x)
    close(y, values(qa), values(b), dtype)
    # same codes: only the order of the sum may differ from the packed call's
    y2 = gpu_lib.mx4_matmul(qa, b, out_dtype=dtype)
    close(y2, values(qa), values(b), dtype)


def test_non_finite_blocks_stay_in_their_rows(gpu_lib):
    """A NaN scale makes its row of the product NaN and no other; K ends
    inside a stage, so the padding behind it must not either."""
    for M, N, K in ((8, 72, 96), (130, 72, 288), (300, 264, 544)):
        a, b = operand(M, K, 1), operand(N, K, 2)
        a[1][M // 2, K // 32 - 1] = 255
        b[1][5, 0] = 255
        b[1][N - 1, K // 32 - 1] = 255
        nan = torch.isnan(gpu_lib.mx4_matmul(a, b, out_dtype=torch.float32))
        want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        want[M // 2] = True
        want[:, [5, N - 1]] = True
        assert torch.equal(nan, want), (M, N, K)


def test_scale_extremes(gpu_lib):
    """Scale bytes 0 and 254 of one operand against their opposites of the
    other: the products are ordinary numbers."""
    for M in (4, 80):
        a, b = operand(M, 64, 3), operand(16, 64, 4)
        a[1].fill_(0)
        b[1].fill_(254)
        y = gpu_lib.mx4_matmul(a, b, out_dtype=torch.float32)
        close(y, values(a), values(b), torch.float32)


def test_product_with_itself_and_shared_inputs(gpu_lib):
    a = operand(64, 256, 6)
    y = gpu_lib.mx4_matmul(a, a, out_dtype=torch.float32)
    close(y, values(a), values(a), torch.float32)


@pytest.mark.parametrize("T,C,K", [(1, 64, 32), (1, 4096, 4096), (7, 200, 96), (40, 64, 576), (64, 136, 256),
                                   (65, 72, 32), (200, 520, 288), (300, 1024, 512), (2050, 2064, 96), (4100, 4160, 256), (130, 1032, 288),
                                   (200, 1000, 512), (4100, 4160, 288),
                                   (300, 1032, 2560), (1200, 2056, 1024), (2100, 2304, 512), (4100, 4160, 1024)])
def test_write_back(gpu_lib, T, C, K):
    print(f"write back T={T} C={C} K={K}", flush=True)
    a, b = operand(T, K, T), operand(C, K, C)
    x = rand((T, 4, C), 7)
    post, res = torch.rand(T, 4, device="cuda"), torch.softmax(rand((T, 4, 4), 8, torch.float32), -1)
    buf = torch.full((T + 1, 4, C), 5.0, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    y = gpu_lib.mx4_write_back(a, b, x, post, res, out=buf[:T], f_out=f)
    va, vb = values(a), values(b)
    close(f, va, vb, torch.bfloat16, "f")
    assert torch.equal(f, gpu_lib.mx4_matmul(a, b))
    F, mF = va @ vb.t(), va.abs() @ vb.abs().t()
    xd, pd, rd = x.double(), post.double()[:, :, None], res.double()
    ref = pd * F[:, None] + torch.matmul(rd, xd)
    mag = pd * F.abs()[:, None] + torch.matmul(rd, xd.abs())
    # f's bar, five roundings of the combination, one of the output
    bound = pd * ((K / 32 + 40) * U * mF)[:, None] + 5 * U * mag + 2.0 ** -8 * ref.abs()
    assert bool(((y.double() - ref).abs() <= bound).all())
    assert bool((buf[T:] == 5.0).all())
    assert torch.equal(y, gpu_lib.mx4_write_back(a, b, x, post, res))  # f_out left out


@pytest.mark.parametrize("T,C", [(1, 64), (1, 7168), (5, 64), (17, 192), (300, 576), (2048, 128), (2049, 128),
                                 (3000, 320), (600, 2112), (2300, 2048)])
@pytest.mark.parametrize("solver", ["newton", "sinkhorn"])
def test_layer_read(gpu_lib, T, C, solver):
    print(f"layer read T={T} C={C} {solver}", flush=True)
    x, Wt = rand((T, 4, C), T), rand((24, 4 * C), C, scale=2.0 / (4 * C) ** 0.5)
    r = gpu_lib.layer_read(x, Wt, solver=solver)
    q = gpu_lib.layer_read(x, Wt, solver=solver, mx4=True, keep_u=True)
    only = gpu_lib.layer_read(x, Wt, solver=solver, mx4=True)
    for k in ("rms", "logits", "H_pre", "H_post", "H_res"):
        assert torch.equal(r[k], q[k]) and torch.equal(r[k], only[k]), k
    assert torch.equal(q["u_values"], r["u"]) and "u_values" not in only
    codes, scales = gpu_lib.mx4_quantize(r["u"])
    for t in (q, only):
        assert torch.equal(t["u"][0], codes) and torch.equal(t["u"][1], scales)
    if T > (8192 if C >= 2048 else 2048):  # the maps pass of the layer forward itself
        fw = gpu_lib.layer_fwd(x, Wt, rand((T, C), 9), solver=solver)
        for k in r:
            assert torch.equal(r[k], fw[k]), k
    xd = x.double().view(T, -1)
    rms = torch.sqrt((xd * xd).mean(1) + 1e-6)
    assert bool(((r["rms"].double() - rms).abs() <= 1e-6 * rms).all())
    logits = xd @ Wt.double().t() / rms[:, None]
    # the logits' bar of the layer (a 4C-term fp32 sum as a random walk)
    S2 = torch.sqrt((xd * xd) @ (Wt.double() ** 2).t()) / rms[:, None]
    lbar = 1e-5 * logits.abs() + 4 * U * (4 * C) ** 0.5 * S2
    assert bool(((r["logits"].double() - logits).abs() <= lbar).all())
    own = r["logits"].double()
    sig = torch.sigmoid(own)
    assert bool(((r["H_pre"].double() - sig[:, :4]).abs() <= 1e-6).all())
    assert bool(((r["H_post"].double() - sig[:, 4:8]).abs() <= 1e-6).all())
    if solver == "newton":
        ref = birkhoff_project(own[:, 8:].reshape(T, 4, 4).cpu().numpy())
        assert np.abs(r["H_res"].cpu().numpy() - ref).max() <= 1e-5
    u = (r["H_pre"].double()[:, :, None] * x.double()).sum(1)
    mag = (r["H_pre"].double()[:, :, None] * x.double().abs()).sum(1)
    assert bool(((r["u"].double() - u).abs() <= 2.0 ** -8 * u.abs() + 5 * U * mag).all())


@pytest.mark.parametrize("M,N,K", [(32, 32, 32), (96, 160, 224), (320, 64, 512)])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_linear_gradients(gpu_lib, M, N, K, fmt):
    """Output and gradients against the formulas: each product of operands
    quantised along its summed axis."""
    for dt in (torch.bfloat16, torch.float32):
        x = rand((M, K), 1, dt).requires_grad_(True)
        w = rand((N, K), 2, dt, 0.1).requires_grad_(True)
        gy = rand((M, N), 3, dt)
        y = gpu_lib.mx4_linear(x, w, format=fmt)
        gx, gw = torch.autograd.grad(y, (x, w), gy)
        f64 = lambda t: t.detach().float().cpu().numpy().astype(np.float64)
        Q = lambda t: torch.from_numpy(K_.quantise(np.ascontiguousarray(t), "e2m1")[2]).cuda()
        xh = K_.quantise(f64(x), fmt)[2]
        close(y.detach(), Q(f64(x)), Q(f64(w)), dt, "y")
        close(gx, Q(f64(gy)), Q(f64(w).T), dt, "grad_x")
        close(gw, Q(f64(gy).T), Q(xh.T), dt, "grad_w")


def test_linear_wanted_gradients(gpu_lib):
    """Each gradient alone is what both together give; no rows give zeros."""
    x, w, gy = rand((96, 64), 1), rand((160, 64), 2), rand((96, 160), 3)
    xr, wr = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    gx, gw = torch.autograd.grad(gpu_lib.mx4_linear(xr, wr), (xr, wr), gy)
    assert torch.equal(torch.autograd.grad(gpu_lib.mx4_linear(xr, w), xr, gy)[0], gx)
    assert torch.equal(torch.autograd.grad(gpu_lib.mx4_linear(x, wr), wr, gy)[0], gw)
    a = rand((96, 64), 4).requires_grad_(True)  # one tensor in both places
    p, q = (a.detach().clone().requires_grad_(True) for _ in range(2))
    ga = torch.autograd.grad(gpu_lib.mx4_linear(a, a), a, gy[:, :96].contiguous())[0]
    gp, gq = torch.autograd.grad(gpu_lib.mx4_linear(p, q), (p, q), gy[:, :96].contiguous())
    assert torch.equal(ga, gp + gq)
    x0 = x[:0].clone().requires_grad_(True)
    g0, w0 = torch.autograd.grad(gpu_lib.mx4_linear(x0, wr).sum(), (x0, wr))
    assert g0.shape == (0, 64) and not bool(w0.any())


def test_linear_strides_and_refusals(gpu_lib):
    """Strided operands and gradients count by value; a second derivative, a
    weight changed in place and wrong tensors raise."""
    x, w, gy = rand((96, 64), 1), rand((160, 64), 2), rand((96, 160), 3)
    ref = [t.clone().requires_grad_(True) for t in (x, w)]
    y = gpu_lib.mx4_linear(*ref)
    want = torch.autograd.grad(y, ref, gy)
    odd = [t.t().contiguous().t().requires_grad_(True) for t in (x, w)]
    got = torch.autograd.grad(gpu_lib.mx4_linear(*odd), odd, gy.t().contiguous().t())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = gpu_lib.mx4_linear(*ref)
    first = torch.autograd.grad(y, ref, gy, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, want))
    with pytest.raises(RuntimeError, match="once"):
        (first[0].float().sum() + first[1].float().sum()).backward()
    y = gpu_lib.mx4_linear(*ref)
    with torch.no_grad():
        ref[1].mul_(2.0)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    for a, b in ((x.cpu(), w), (x, w.cpu()), (x.half(), w), (x, w.double())):
        with pytest.raises((TypeError, ValueError)):
            gpu_lib.mx4_linear(a, b)
    with pytest.raises(ValueError):
        gpu_lib.mx4_linear(x, rand((160, 96), 2))
    with pytest.raises(ValueError):
        gpu_lib.mx4_linear(x[:95], w)
    assert not gpu_lib.mx4_linear(x, w).requires_grad


def test_linear_captured(gpu_lib):
    """A training step recorded in a graph, its gradients written by value, on
    every replay what the eager step gives; and inference mode."""
    x, w, gy = rand((96, 64), 1), rand((160, 64), 2), rand((96, 160), 3)
    leaves = [t.clone().requires_grad_(True) for t in (x, w)]
    out = []

    def step():
        y = gpu_lib.mx4_linear(*leaves)
        return [y.detach(), *torch.autograd.grad(y, leaves, gy)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        with torch.no_grad():
            leaves[0].copy_(rand((96, 64), 10 + k))
            leaves[1].copy_(rand((160, 64), 20 + k))
        gy.copy_(rand((96, 160), 30 + k))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        fresh = [t.detach().clone().requires_grad_(True) for t in leaves]
        y = gpu_lib.mx4_linear(*fresh)
        want = [y.detach(), *torch.autograd.grad(y, fresh, gy)]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
    with torch.inference_mode():
        assert torch.equal(gpu_lib.mx4_linear(*[t.detach().clone() for t in leaves]), want[0])


def test_captured_backward_of_an_eager_graph_raises(gpu_lib):
    """While an eager graph of the same leaves lives, a captured backward is
    refused in the node before the one it could not reach; without it the same
    capture goes through."""
    gy = rand((64, 96), 3)
    x, w = rand((64, 32), 1).requires_grad_(True), rand((96, 32), 2).requires_grad_(True)
    xm = rand((4, 4, 64), 4).requires_grad_(True)
    lg = rand((4, 4, 4), 5, torch.float32).requires_grad_(True)
    gm = rand((4, 4, 64), 6)
    cases = [lambda: torch.autograd.grad(gpu_lib.mx4_linear(x, w), (x, w), gy),
             lambda: torch.autograd.grad(gpu_lib.projected_mix(xm, lg), (xm, lg), gm)]
    held = [gpu_lib.mx4_linear(x, w), gpu_lib.projected_mix(xm, lg)]
    torch.cuda.synchronize()
    for run in cases:
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="eager graph"):
            with torch.cuda.graph(graph):
                run()
        torch.cuda.synchronize()
    del held
    for run in cases:
        want = run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_linear_gradient_by_differences(gpu_lib):
    """With operands that MXFP4 and the checkpoint hold exactly, the map is
    bilinear and a central difference of the loss is its derivative."""
    M = N = K = 64
    g = torch.Generator().manual_seed(7)
    small = lambda: torch.randint(-2, 3, (64, 64), generator=g).float().cuda()
    x, w, gy = small().requires_grad_(True), small().requires_grad_(True), small()
    with torch.no_grad():  # every block of 32, along either axis, holds exactly
        for t in (x, w, gy):
            t[:, ::32], t[::32, :] = 2.0, 2.0
    gx, gw = torch.autograd.grad(gpu_lib.mx4_linear(x, w), (x, w), gy)
    d = torch.zeros_like(x)
    d[5, 9] = 1.0
    for t, grad in ((x, gx), (w, gw)):
        loss = lambda e: float((((x + e * d) if t is x else x).detach().double() @ ((w + e * d) if t is w else w).detach().double().t()
                                * gy.double()).sum())
        assert abs((loss(0.5) - loss(-0.5)) - float(grad[5, 9])) <= 1e-9


def test_sublayer_run(gpu_lib):
    """Read, two products and write-back as they are used together, for one
    token and for many, eagerly, replayed from a graph and on another
    stream."""
    for T in (1, 130, 2100):
        C, H = 256, 512
        x, Wt = rand((T, 4, C), 20), rand((24, 4 * C), 21, scale=2.0 / (4 * C) ** 0.5)
        up = gpu_lib.mx4_quantize(rand((H, C), 22, scale=C ** -0.5))
        down = gpu_lib.mx4_quantize(rand((C, H), 23, scale=H ** -0.5))

        def run():
            r = gpu_lib.layer_read(x, Wt, mx4=True)
            h = torch.relu(gpu_lib.mx4_matmul(r["u"], up))
            hq = gpu_lib.mx4_quantize(h)
            out = gpu_lib.mx4_write_back(hq, down, x, r["H_post"], r["H_res"])
            return out, h, hq[0], r["H_post"], r["H_res"], *r["u"]

        want = [t.clone() for t in run()]
        out, h, _, post, res, uc, us = want
        hq = gpu_lib.mx4_quantize(h)
        F = values(hq) @ values(down).t()
        ref = post.double()[:, :, None] * F[:, None] + torch.matmul(res.double(), x.double())
        mag = post.double()[:, :, None] * (values(hq).abs() @ values(down).abs().t())[:, None] \
            + torch.matmul(res.double(), x.double().abs())
        assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (H / 32 + 45) * U * mag).all())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for rep in range(4):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (T, rep)
            run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = run()
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), T


def test_binding_refuses_what_does_not_fit(gpu_lib):
    a, b = operand(16, 64, 1), operand(32, 64, 2)
    x, post, res = rand((16, 4, 32), 3), rand((16, 4), 4, torch.float32), rand((16, 4, 4), 5, torch.float32)
    out = torch.full((16, 32), 9.0, dtype=torch.bfloat16, device="cuda")
    bad = [lambda: gpu_lib.mx4_matmul(a, operand(32, 96, 3)), lambda: gpu_lib.mx4_matmul((a[0], a[1][:-1]), b),
           lambda: gpu_lib.mx4_matmul(a, b, out=out[:-1]), lambda: gpu_lib.mx4_matmul(rand((16, 32), 6), b),
           lambda: gpu_lib.mx4_write_back(a, b, x[:-1], post, res), lambda: gpu_lib.mx4_write_back(b, a, x, post, res),
           lambda: gpu_lib.mx4_write_back(a, b, x, post[:-1], res),
           lambda: gpu_lib.mx4_write_back(a, b, x, post, res, f_out=out[:-1]),
           lambda: gpu_lib.layer_read(rand((4, 4, 64), 1), rand((24, 128), 2)),
           lambda: gpu_lib.mx4_dequantize(a[0], b[1])]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", k)
    with pytest.raises(gpu_lib.MHCError):
        gpu_lib.mx4_matmul(a, operand(12, 64, 3))
    torch.cuda.synchronize()
    assert bool((out == 9.0).all())
    e = gpu_lib.mx4_matmul((a[0][:0], a[1][:0]), b)
    assert e.shape == (0, 32)
