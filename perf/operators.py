"""The activation-checkpoint and microscaled 4-bit operators as workloads.

Each case is one pass through an operator as a training or serving program
calls it.  ``run`` computes it either through the package (``own`` true) or in
its plain form: elementary torch operations in 32 bits (64 for the map
projections, whose solves lose digits in 32), rounded once at the end.
``exact`` computes the same outputs in 64 bits, written apart from the plain
form.

The operators (formats: blocks of 32 along the last axis with one power-of-two
scale each; elements e4m3, int8 in units of scale/64, or e2m1):

ckpt        an activation packed to an 8-bit checkpoint and read back
mix         a training step of the stream mix that keeps x as a checkpoint:
            out = H x, then grad_x = H^T g and grad_H = g xhat^T
layer       a training step of the residual layer that keeps x and f as
            checkpoints
quant       quantisation to MXFP4, along the rows or (transposed) along the
            columns, and the values it stands for
matmul      a linear map whose operands are both MXFP4: a serving call on
            activations and packed weights, or a training step
sublayer    the read half of the layer, an MXFP4 product as the layer
            function, and the write-back in the product's epilogue
"""
import math

import torch

own = False

BLOCK = 32
EPS = 1e-6
# largest element and smallest scale byte of each element format (the smallest
# byte keeps every stored value zero or a normal fp32 and bf16 number)
FORMATS = {"e4m3": (448.0, 10), "int8": (127.0 / 64.0, 7), "e2m1": (6.0, 2)}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's four streams: what a latency-bound caller packs
        dict(name="ckpt_token", op="ckpt", R=4, C=4096, fmt="int8", dtype="bf16"),
        # the layer-function outputs of the full-size layer step
        dict(name="ckpt_full", op="ckpt", R=65536, C=7168, fmt="e4m3", dtype="bf16"),
        # a short ragged batch: width not a multiple of the block
        dict(name="mix_ragged", op="mix", T=241, C=520, fmt="int8"),
        # the stream-mix workload's size
        dict(name="mix_16384x4096", op="mix", T=16384, C=4096, fmt="e4m3"),
        # a small layer, token count off every tile
        dict(name="layer_small", op="layer", T=300, C=256, fmt="int8"),
        # the full layer width, a quarter of the full step's tokens
        dict(name="layer_16384x7168", op="layer", T=16384, C=7168, fmt="e4m3"),
        # one decoded token's layer input
        dict(name="quant_token", op="quant", R=1, C=7168, dtype="bf16", transpose=False),
        # a gradient quantised along its tokens for the weight gradient
        dict(name="quant_grad_t", op="quant", R=16384, C=7168, dtype="bf16", transpose=True),
        # serving, one token: bound by the packed weights
        dict(name="matmul_token", op="matmul", mode="serve", M=1, N=7168, K=7168, dtype="bf16"),
        # training step of a linear map, three products
        dict(name="matmul_train", op="matmul", mode="train", M=8192, N=8192, K=4096, dtype="bf16"),
        # serving, one token through read, product and write-back
        dict(name="sublayer_token", op="sublayer", T=1, C=4096),
        # a long prefill through the same
        dict(name="sublayer_16384x4096", op="sublayer", T=16384, C=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ckpt", "mix", "layer", "quant", "matmul", "sublayer"])
    if op == "ckpt":
        C = 8 * _log_int(rng, 1, 1024)
        R = _log_int(rng, 1, max(1, min(262144, 65536 * 7168 // C)))
        return dict(op=op, R=R, C=C, fmt=rng.choice(["e4m3", "int8"]),
                    dtype=rng.choice(["bf16", "f32"]) if R * C <= 1 << 28 else "bf16")
    if op == "mix":
        C = 8 * _log_int(rng, 1, 896)
        return dict(op=op, T=_log_int(rng, 1, min(65536, 16384 * 4096 // C)), C=C,
                    fmt=rng.choice(["e4m3", "int8"]))
    if op == "layer":
        C = 64 * _log_int(rng, 1, 112)
        return dict(op=op, T=_log_int(rng, 1, min(65536, 16384 * 7168 // C)), C=C,
                    fmt=rng.choice(["e4m3", "int8"]))
    if op == "quant":
        transpose = rng.random() < 0.5
        R = 32 * _log_int(rng, 1, 1024) if transpose else _log_int(rng, 1, 32768)
        C = 32 * _log_int(rng, 1, min(512, max(1, 16384 * 7168 // R // 32)))
        return dict(op=op, R=R, C=C, dtype=rng.choice(["bf16", "f32"]) if R * C <= 1 << 26 else "bf16",
                    transpose=transpose)
    if op == "matmul":
        if rng.random() < 0.5:
            return dict(op=op, mode="serve", M=_log_int(rng, 1, 4096), N=8 * _log_int(rng, 16, 1024),
                        K=32 * _log_int(rng, 4, 256), dtype=rng.choice(["bf16", "f32"]))
        return dict(op=op, mode="train", M=32 * _log_int(rng, 1, 256), N=32 * _log_int(rng, 4, 256),
                    K=32 * _log_int(rng, 4, 128), dtype="bf16")
    C = 64 * _log_int(rng, 1, 64)
    return dict(op=op, T=_log_int(rng, 1, 16384), C=C)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


class _Draws:
    """Seeded draws on the GPU, made in pieces so that the fp32 staging of a
    large bf16 tensor stays small."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def normal(self, shape, scale=1.0):
        return torch.randn(shape, generator=self.gen, device="cuda") * scale

    def rows(self, R, C, dtype, columns=None):
        """[R, C] normal values, each column times its own factor."""
        out = torch.empty((R, C), dtype=dtype, device="cuda")
        step = max(1, (1 << 27) // C)
        for r in range(0, R, step):
            t = torch.randn((min(step, R - r), C), generator=self.gen, device="cuda")
            if columns is not None:
                t *= columns
            out[r:r + step] = t
        return out

    def activations(self, R, C, dtype=torch.bfloat16):
        """Residual-stream-like rows: log-normal channel sizes, and one
        channel in 256 twenty times larger."""
        col = torch.exp(0.5 * self.normal((C,)))
        out = torch.rand((C,), generator=self.gen, device="cuda") < 1.0 / 256.0
        return self.rows(R, C, dtype, torch.where(out, 20.0 * col, col))


def _doubly_stochastic(d, T):
    """[T,4,4] fp32 mixing matrices: N(0,1) logits scaled to unit row and
    column sums."""
    P = torch.exp(d.normal((T, 4, 4)).double())
    for _ in range(100):
        P = P / P.sum(-1, keepdim=True)
        P = P / P.sum(-2, keepdim=True)
    return P.float()


def prepare(case, seed):
    d = _Draws(seed)
    op = case["op"]
    s = {"case": case}
    if op == "ckpt":
        s["x"] = d.activations(case["R"], case["C"], _dtype(case["dtype"]))
    elif op == "mix":
        T, C = case["T"], case["C"]
        s["x"] = d.activations(4 * T, C).view(T, 4, C)
        s["g"] = d.rows(4 * T, C, torch.bfloat16).view(T, 4, C)
        s["H"] = _doubly_stochastic(d, T)
    elif op == "layer":
        T, C = case["T"], case["C"]
        s["x"] = d.rows(4 * T, C, torch.bfloat16).view(T, 4, C)
        s["W"] = d.normal((24, 4 * C), 1.0 / math.sqrt(4 * C)).bfloat16()
        s["f"] = d.rows(T, C, torch.bfloat16)
        s["gxo"] = d.rows(4 * T, C, torch.bfloat16).view(T, 4, C)
        s["gu"] = d.rows(T, C, torch.bfloat16)
        if own:
            import birkhoff_projection_amd as bp
            s["workspace"] = bp.layer_ckpt_workspace(T, C, s["x"].device)
    elif op == "quant":
        s["x"] = d.activations(case["R"], case["C"], _dtype(case["dtype"]))
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        w = d.normal((N, K), 1.0 / math.sqrt(K))
        s["x"] = d.activations(M, K, _dtype(case["dtype"]))
        if case["mode"] == "serve":
            s["w"] = _mx4_pack(w)
        else:
            s["w"] = w.bfloat16()
            s["gy"] = d.rows(M, N, torch.bfloat16)
    else:
        T, C = case["T"], case["C"]
        s["x"] = d.rows(4 * T, C, torch.bfloat16).view(T, 4, C)
        s["W"] = d.normal((24, 4 * C), 1.0 / math.sqrt(4 * C)).bfloat16()
        s["w"] = _mx4_pack(d.normal((C, C), 1.0 / math.sqrt(C)))
    return s


def _mx4_pack(w):
    """MXFP4 weights as a file holds them: codes [N, K/2] (even elements in
    the low half of a byte) and scale bytes [N, K/32]."""
    N, K = w.shape
    byte = _scale_bytes(w.float().view(N, K // BLOCK, BLOCK), "e2m1")
    v = w.float().view(N, K // BLOCK, BLOCK) / _power(byte)
    a = _round_e2m1(v).abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).view(N, K)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), byte.view(N, K // BLOCK).to(torch.uint8)


# ---------------------------------------------------------------------------
# plain forms, 32 bits
# ---------------------------------------------------------------------------

def _scale_bytes(blocks, fmt):
    """Smallest b with max|block| <= largest * 2^(b - 127), by the bits of the
    fp32 maximum; [..., blocks, 1] int32."""
    largest, lo = FORMATS[fmt]
    frac, exp = math.frexp(largest)  # largest = frac 2^exp, frac in [1/2, 1)
    carry = (1 << 23) - 1 - int((2 * frac - 1) * (1 << 23))
    amax = blocks.abs().amax(-1, keepdim=True)
    b = ((amax.view(torch.int32) + carry) >> 23) - (exp - 1)
    return b.clamp(lo, 254)


def _power(byte):
    """2^(byte - 127) as fp32."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _round_e2m1(v):
    """|v| <= 6 to the nearest e2m1 value, ties to the even code."""
    a = v.abs()
    q = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(v / q) * q


def _round_e4m3(v):
    """|v| <= 448 to the nearest e4m3 value, ties to the even code."""
    e = ((v.abs().view(torch.int32) >> 23) - 127).clamp(min=-6)
    q = _power(e - 3 + 127)
    return torch.round(v / q) * q


def _round_int8(v):
    return torch.round(v * 64.0).clamp(-127, 127) / 64.0


_ROUND = {"e4m3": _round_e4m3, "int8": _round_int8, "e2m1": _round_e2m1}


def _quantised(x, fmt):
    """fp32 values that x stands for after packing along its last axis."""
    C = x.shape[-1]
    x = x.float()
    pad = -C % BLOCK
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    v = x.reshape(x.shape[:-1] + (-1, BLOCK))
    p = _power(_scale_bytes(v, fmt))
    y = (_ROUND[fmt](v / p) * p).reshape(x.shape)
    return y[..., :C] if pad else y


def _mx4_values(codes, scales):
    """fp32 values of MXFP4 codes [N, K/2] and scale bytes [N, K/32]."""
    N = codes.shape[0]
    c = torch.stack((codes & 15, codes >> 4), dim=-1).view(N, -1, BLOCK)
    m = (c & 7).float()
    a = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(c > 7, -a, a) * _power(scales.to(torch.int32)).unsqueeze(-1)
    return v.view(N, -1)


def _project(logits):
    """Doubly stochastic scaling of exp(logits) [T,4,4] in 64 bits: ten
    Sinkhorn sweeps, then Newton on the three free column potentials."""
    a = logits.double()
    a = a - a.amax(-1, keepdim=True)
    P = torch.exp(a)
    for _ in range(10):
        P = P / P.sum(-1, keepdim=True)
        P = P / P.sum(-2, keepdim=True)
    for _ in range(6):
        P = P / P.sum(-1, keepdim=True)
        c = P.sum(-2)
        beta = _laplacian_solve(P, (1.0 - c)[:, :3])
        P = P * torch.exp(torch.nn.functional.pad(beta, (0, 1))).unsqueeze(-2)
    return P / P.sum(-1, keepdim=True)


def _laplacian_solve(P, r):
    """beta [T,3] of (diag - P^T P) beta = r with the fourth potential fixed;
    the diagonal is the sum of the off-diagonal weights."""
    w = (P.unsqueeze(-1) * P.unsqueeze(-2)).sum(1)
    w01, w02, w12 = w[:, 0, 1], w[:, 0, 2], w[:, 1, 2]
    a = w01 + w02 + w[:, 0, 3]
    b = w01 + w12 + w[:, 1, 3]
    c = w02 + w12 + w[:, 2, 3]
    m00, m01, m02 = b * c - w12 * w12, w01 * c + w02 * w12, w01 * w12 + w02 * b
    m11, m12, m22 = a * c - w02 * w02, a * w12 + w01 * w02, a * b - w01 * w01
    det = a * m00 - w01 * m01 - w02 * m02
    r0, r1, r2 = r[:, 0], r[:, 1], r[:, 2]
    return torch.stack((m00 * r0 + m01 * r1 + m02 * r2, m01 * r0 + m11 * r1 + m12 * r2,
                        m02 * r0 + m12 * r1 + m22 * r2), dim=-1) / det.unsqueeze(-1)


def _project_bwd(P, G):
    """dL/dlogits [T,4,4] from P and dL/dP, in 64 bits."""
    P, G = P.double(), G.double()
    a = (P * G).sum(-1, keepdim=True)
    r = (P * (G - a)).sum(-2)[:, :3]
    beta = torch.nn.functional.pad(_laplacian_solve(P, r), (0, 1)).unsqueeze(-2)
    h = G - beta
    return P * (h - (P * h).sum(-1, keepdim=True))


def _maps(x, W):
    """The layer's per-token maps in 32 bits (the projection in 64)."""
    T, n, C = x.shape
    xf = x.view(T, 4 * C).float()
    rms = torch.sqrt((xf * xf).mean(-1) + EPS)
    logits = (xf @ W.float().t()) / rms.unsqueeze(-1)
    H_res = _project(logits[:, 8:].view(T, 4, 4)).float()
    return dict(rms=rms, logits=logits, H_pre=torch.sigmoid(logits[:, :4]),
                H_post=torch.sigmoid(logits[:, 4:8]), H_res=H_res)


def _combine(H, x):
    """sum_j H[t,i,j] x[t,j,:] stream by stream (x fp32 or narrower)."""
    return torch.stack([sum(H[:, i, j, None] * x[:, j].float() for j in range(x.shape[1]))
                        for i in range(H.shape[1])], dim=1)


def _dots(g, x):
    """[T,i,j] dot products of the streams g[t,i,:] and x[t,j,:]."""
    return torch.stack([torch.stack([(g[:, i].float() * x[:, j].float()).sum(-1)
                                     for j in range(x.shape[1])], -1) for i in range(g.shape[1])], 1)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "ckpt":
        return _quantised(s["x"], case["fmt"]).to(s["x"].dtype)
    if op == "mix":
        xh = _quantised(s["x"], case["fmt"])
        return (_combine(s["H"], s["x"]).bfloat16(), _combine(s["H"].transpose(1, 2), s["g"]).bfloat16(),
                _dots(s["g"], xh))
    if op == "layer":
        return _plain_layer(s)
    if op == "quant":
        x = s["x"].t() if case["transpose"] else s["x"]
        return _quantised(x.contiguous(), "e2m1").to(s["x"].dtype)
    if op == "matmul":
        if case["mode"] == "serve":
            return (_quantised(s["x"], "e2m1") @ _mx4_values(*s["w"]).t()).to(s["x"].dtype)
        x, w, gy = s["x"], s["w"], s["gy"]
        y = _quantised(x, "e2m1") @ _quantised(w, "e2m1").t()
        gx = _quantised(gy, "e2m1") @ _quantised(w.t().contiguous(), "e2m1").t()
        xh = _quantised(x, "e4m3")
        gw = _quantised(gy.t().contiguous(), "e2m1") @ _quantised(xh.t().contiguous(), "e2m1").t()
        return y.bfloat16(), gx.bfloat16(), gw.bfloat16()
    x = s["x"]
    m = _maps(x, s["W"])
    u = _combine(m["H_pre"].unsqueeze(1), x)[:, 0].bfloat16()
    f = _quantised(u, "e2m1") @ _mx4_values(*s["w"]).t()
    out = _combine(m["H_res"], x) + m["H_post"].unsqueeze(-1) * f.unsqueeze(1)
    return out.bfloat16(), m["H_pre"], m["H_post"], m["H_res"]


def _plain_layer(s):
    x, W, f, gxo, gu = s["x"], s["W"], s["f"], s["gxo"], s["gu"]
    T, n, C = x.shape
    m = _maps(x, W)
    u = _combine(m["H_pre"].unsqueeze(1), x)[:, 0]
    out = _combine(m["H_res"], x) + m["H_post"].unsqueeze(-1) * f.float().unsqueeze(1)
    u, out = u.bfloat16(), out.bfloat16()
    xh, fh = _quantised(x, s["case"]["fmt"]), _quantised(f, s["case"]["fmt"])
    d_pre = _dots(gu.unsqueeze(1), xh)[:, 0]
    d_post = _dots(gxo, fh.unsqueeze(1))[:, :, 0]
    dl = torch.cat((d_pre * m["H_pre"] * (1 - m["H_pre"]), d_post * m["H_post"] * (1 - m["H_post"]),
                    _project_bwd(m["H_res"], _dots(gxo, xh)).float().view(T, 16)), dim=1)
    inv = (1.0 / m["rms"]).unsqueeze(-1)
    share = ((dl * m["logits"]).sum(-1, keepdim=True) / (4 * C)) * inv
    gf = (m["H_post"].unsqueeze(-1) * gxo.float()).sum(1)
    xh = xh.view(T, 4 * C)
    gW = (dl * inv).t() @ xh
    gx = (dl @ W.float() - xh * share) * inv
    gx = gx.view(T, 4, C) + _combine(m["H_res"].transpose(1, 2), gxo)
    gx = gx + m["H_pre"].unsqueeze(-1) * gu.float().unsqueeze(1)
    return dict(u=u, x_out=out, grad_x=gx.bfloat16(), grad_f=gf.bfloat16(), grad_W=gW, grad_logits=dl)


# ---------------------------------------------------------------------------
# through the package
# ---------------------------------------------------------------------------

def _through_package(s):
    import birkhoff_projection_amd as bp
    case = s["case"]
    op = case["op"]
    if op == "ckpt":
        codes, scales = bp.ckpt_pack(s["x"], format=case["fmt"])
        return bp.ckpt_unpack(codes, scales, format=case["fmt"], dtype=s["x"].dtype)
    if op == "mix":
        out, ckpt = bp.stream_mix_ckpt(s["x"], s["H"], format=case["fmt"])
        gx, gH = bp.stream_mix_bwd_ckpt(ckpt, s["H"], s["g"], format=case["fmt"])
        return out, gx, gH
    if op == "layer":
        fwd, ckpt = bp.layer_fwd_ckpt(s["x"], s["W"], s["f"], format=case["fmt"])
        g = bp.layer_bwd_ckpt(ckpt, s["W"], fwd, s["gxo"], s["gu"], format=case["fmt"],
                              workspace=s["workspace"])
        return dict(u=fwd["u"], x_out=fwd["x_out"], grad_x=g["grad_x"], grad_f=g["grad_f"],
                    grad_W=g["grad_W"], grad_logits=g["grad_logits"])
    if op == "quant":
        codes, scales = bp.mx4_quantize(s["x"], transpose=case["transpose"])
        return bp.mx4_dequantize(codes, scales, dtype=s["x"].dtype)
    if op == "matmul":
        if case["mode"] == "serve":
            return bp.mx4_matmul(s["x"], s["w"], out_dtype=s["x"].dtype)
        x, w = s["x"].requires_grad_(True), s["w"].requires_grad_(True)
        y = bp.mx4_linear(x, w)
        gx, gw = torch.autograd.grad(y, (x, w), s["gy"])
        return y.detach(), gx, gw
    r = bp.layer_read(s["x"], s["W"], mx4=True)
    out = bp.mx4_write_back(r["u"], s["w"], s["x"], r["H_post"], r["H_res"])
    return out, r["H_pre"], r["H_post"], r["H_res"]


def run(state):
    return _through_package(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# work: each input read once, each output written once
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "ckpt":
        e = case["R"] * case["C"]
        w = 2 if case["dtype"] == "bf16" else 4
        packed = e + case["R"] * -(-case["C"] // BLOCK)
        return {"bytes": 2 * (e * w + packed), "flops": 4 * e}
    if op == "mix":
        T, C = case["T"], case["C"]
        e = 4 * T * C
        packed = e + 4 * T * -(-C // BLOCK)
        return {"bytes": e * 2 * 4 + 2 * packed + 3 * 64 * T, "flops": 3 * 8 * e}
    if op == "layer":
        T, C = case["T"], case["C"]
        e = T * C
        packed = 5 * (e + e // BLOCK)
        maps = T * (1 + 24 + 8 + 16) * 4
        # forward: x, f in; u, x_out and the checkpoint out; backward: the
        # checkpoint, grad_x_out and grad_u in; grad_x and grad_f out
        data = 2 * e * (4 + 1 + 1 + 4) + 2 * packed + 2 * e * (4 + 1 + 4 + 1)
        return {"bytes": data + 2 * maps + T * 96 + 2 * 24 * 4 * C * 2 + 24 * 4 * C * 4,
                "flops": e * (3 * 2 * 24 * 4 + 2 * 20 + 2 * 24 + 2 * 24)}
    if op == "quant":
        e = case["R"] * case["C"]
        w = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * (e * w + e // 2 + e // BLOCK), "flops": 4 * e}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        w = 2 if case["dtype"] == "bf16" else 4
        if case["mode"] == "serve":
            return {"bytes": M * K * w + N * K * 17 // 32 + M * N * w, "flops": 2 * M * N * K}
        return {"bytes": 2 * (2 * M * K + 2 * N * K + 2 * M * N), "flops": 6 * M * N * K}
    T, C = case["T"], case["C"]
    return {"bytes": 2 * 8 * T * C + C * C * 17 // 32 + 24 * 4 * C * 2 + T * 24 * 4,
            "flops": T * C * (2 * 24 * 4 + 2 * C + 2 * 4 + 2 * 20)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _table(fmt):
    """Every non-negative value of an element format, in code order."""
    if fmt == "int8":
        return [i / 64.0 for i in range(128)]
    man, low, top = (3, -6, 448.0) if fmt == "e4m3" else (1, 0, 6.0)
    out, code = [], 0
    while True:
        e, m = divmod(code, 1 << man)
        v = math.ldexp(m, low - man) if e == 0 else math.ldexp((1 << man) + m, low - man + e - 1)
        if v > top:
            return out
        out.append(v)
        code += 1


def _exact_power(e):
    """2^e as a normal double, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quantised(x, fmt):
    """64-bit values of x packed along its last axis, by a search in the
    table of the format's values; worked off in pieces of rows."""
    largest, lo = FORMATS[fmt]
    frac, exp = math.frexp(largest)
    tab = torch.tensor(_table(fmt), dtype=torch.float64, device=x.device)
    mid = (tab[1:] + tab[:-1]) / 2
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    C = x.shape[-1]
    src, dst = x.reshape(-1, C), out.view(-1, C)
    step = max(1, (1 << 25) // C)
    for r in range(0, src.shape[0], step):
        v = src[r:r + step].double()
        v = torch.nn.functional.pad(v, (0, -C % BLOCK)).view(v.shape[0], -1, BLOCK)
        mant, e = torch.frexp(v.abs().amax(-1, keepdim=True))
        p = e - exp + (mant > frac).to(e.dtype)
        p = torch.where(mant == 0, torch.full_like(p, lo - 127), p).clamp(lo - 127, 127)
        a = v.abs() * _exact_power(-p)
        i = torch.searchsorted(mid, a)           # midpoints below a: ties fall to the lower code
        at = i.clamp(max=len(mid) - 1)
        i = i + ((a == mid[at]) & (i < len(mid)) & (i % 2 == 1)).to(i.dtype)
        q = torch.copysign(tab[i], v) * _exact_power(p)
        dst[r:r + step] = q.reshape(v.shape[0], -1)[:, :C]
    return out


def _exact_mx4_values(codes, scales):
    N = codes.shape[0]
    t = _table("e2m1")
    tab = torch.tensor(t + [-v for v in t], dtype=torch.float64, device=codes.device)
    v = torch.empty((N, 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    v[:, 0::2] = tab[(codes % 16).long()]
    v[:, 1::2] = tab[(codes // 16).long()]
    return v * _exact_power(scales.long() - 127).repeat_interleave(BLOCK, dim=1)


def _exact_projection(logits):
    """Sinkhorn sweeps until every row and column sum is 1 to 1e-14."""
    a = logits.double()
    P = torch.softmax(a, -1)
    for _ in range(100):
        for _ in range(50):
            P = P / P.sum(-1, keepdim=True)
            P = P / P.sum(-2, keepdim=True)
        if float((P.sum(-1) - 1).abs().max()) < 1e-14:
            break
    return P


def _exact_projection_bwd(P, G):
    """dA = P o (G - alpha 1' - 1 beta') whose rows and columns sum to zero:
    the 8 linear conditions with beta_3 = 0, solved as one 7 x 7 system."""
    P, G = P.double(), G.double()
    A = torch.zeros(P.shape[0], 7, 7, dtype=torch.float64, device=P.device)
    A[:, :4, :4] = torch.diag_embed(P.sum(2))
    A[:, :4, 4:] = P[:, :, :3]
    A[:, 4:, :4] = P[:, :, :3].transpose(1, 2)
    A[:, 4:, 4:] = torch.diag_embed(P.sum(1)[:, :3])
    y = P * G
    b = torch.cat((y.sum(2), y.sum(1)[:, :3]), dim=1)
    z = torch.linalg.solve(A, b.unsqueeze(-1)).squeeze(-1)
    beta = torch.cat((z[:, 4:], torch.zeros_like(z[:, :1])), dim=1)
    return P * (G - z[:, :4, None] - beta[:, None, :])


def _exact_maps(x, W):
    x = x.double().flatten(1)
    rms = torch.sqrt(x.pow(2).sum(1) / x.shape[1] + EPS)
    logits = (x / rms[:, None]) @ W.double().t()
    sig = 1.0 / (1.0 + torch.exp(-logits[:, :8]))
    return rms, logits, sig[:, :4], sig[:, 4:], _exact_projection(logits[:, 8:].reshape(-1, 4, 4))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ckpt":
        return _exact_quantised(s["x"], case["fmt"])
    if op == "mix":
        x, g, H = s["x"], s["g"].double(), s["H"].double()
        out = torch.matmul(H, x.double())
        return out, torch.matmul(H.transpose(1, 2).contiguous(), g), torch.matmul(
            g, _exact_quantised(x, case["fmt"]).transpose(1, 2).contiguous())
    if op == "layer":
        return _exact_layer(s)
    if op == "quant":
        return _exact_quantised(s["x"].t().contiguous() if case["transpose"] else s["x"], "e2m1")
    if op == "matmul":
        x, w = s["x"], s["w"]
        if case["mode"] == "serve":
            return _exact_quantised(x, "e2m1") @ _exact_mx4_values(*w).t()
        gy = s["gy"]
        xt = _exact_quantised(x, "e4m3").t().contiguous()
        return (_exact_quantised(x, "e2m1") @ _exact_quantised(w, "e2m1").t(),
                _exact_quantised(gy, "e2m1") @ _exact_quantised(w.t().contiguous(), "e2m1").t(),
                _exact_quantised(gy.t().contiguous(), "e2m1") @ _exact_quantised(xt, "e2m1").t())
    x = s["x"]
    _, _, pre, post, res = _exact_maps(x, s["W"])
    # the layer input is defined as a bf16 tensor, which the product quantises
    u = torch.matmul(pre.unsqueeze(1), x.double())[:, 0].bfloat16()
    f = _exact_quantised(u, "e2m1") @ _exact_mx4_values(*s["w"]).t()
    return torch.matmul(res, x.double()) + post[:, :, None] * f[:, None, :], pre, post, res


def _exact_layer(s):
    W, T, C = s["W"].double(), s["x"].shape[0], s["x"].shape[2]
    D = 4 * C
    gW = torch.zeros(24, D, dtype=torch.float64, device=W.device)
    parts = []
    step = max(1, (1 << 27) // D)
    for t in range(0, T, step):
        x, f, go, gu = (s[k][t:t + step].double() for k in ("x", "f", "gxo", "gu"))
        rms, logits, pre, post, res = _exact_maps(s["x"][t:t + step], s["W"])
        u = torch.matmul(pre.unsqueeze(1), x)[:, 0]
        out = torch.matmul(res, x) + post[:, :, None] * f[:, None, :]
        xh = _exact_quantised(s["x"][t:t + step], s["case"]["fmt"])
        fh = _exact_quantised(s["f"][t:t + step], s["case"]["fmt"])
        xt = xh.transpose(1, 2).contiguous()
        dl = torch.cat((torch.matmul(gu.unsqueeze(1), xt)[:, 0] * pre * (1 - pre),
                        torch.matmul(go, fh.unsqueeze(-1))[:, :, 0] * post * (1 - post),
                        _exact_projection_bwd(res, torch.matmul(go, xt)).reshape(-1, 16)), dim=1)
        xn = xh.reshape(-1, D) / rms[:, None]
        gW += dl.t() @ xn
        # through the normalisation: <dl W, x / rms> is <dl, logits>
        gn = (dl @ W - xn * ((dl * logits).sum(1, keepdim=True) / D)) / rms[:, None]
        gx = torch.matmul(res.transpose(1, 2).contiguous(), go) + pre[:, :, None] * gu[:, None, :] \
            + gn.reshape(-1, 4, C)
        gf = torch.matmul(post.unsqueeze(1), go)[:, 0]
        parts.append((u, out, gx, gf, dl))
    u, out, gx, gf, dl = (torch.cat(p) for p in zip(*parts))
    return dict(u=u, x_out=out, grad_x=gx, grad_f=gf, grad_W=gW, grad_logits=dl)
