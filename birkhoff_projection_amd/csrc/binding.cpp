// Marshalling of the checkpoint and 4-bit calls between PyTorch tensors and
// the C ABI (include/mhc.h).
//
// A small call lasts a few microseconds on the GPU, less than the same
// marshalling takes through ctypes and torch's Python front end (7.8 us a call,
// 3 of them in two torch.empty).  So these calls check their tensors, allocate
// their outputs and take the current stream here.  Every function returns the
// ABI's status first (0 = MHC_OK) and then its output tensors; a tensor of the
// wrong type raises TypeError, of the wrong shape, layout or device ValueError,
// before anything is enqueued.
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/utils/pybind.h>

#include <tuple>
#include <unordered_set>
#include <vector>

#include "../../include/mhc.h"

namespace {

using at::Tensor;
using Opt = c10::optional<Tensor>;

constexpr int64_t kBlock = 32;

void need(const Tensor& t, const char* name, at::ScalarType dtype)
{
    TORCH_CHECK_TYPE(t.defined() && t.is_cuda(), name, " must be a CUDA (HIP) tensor");
    TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, " must be ", dtype, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}

// A tensor that the call reads, of exactly this shape on this device.
void given(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
           const at::Device& device)
{
    need(t, name, dtype);
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
    TORCH_CHECK_VALUE(t.device() == device, name, " must be on ", device, ", got ", t.device());
}

// The caller's output buffer, checked as above (a short or misplaced one would
// let a kernel write past its allocation), or a new one.
Tensor output(const Opt& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
              const Tensor& like)
{
    if (!t.has_value()) return at::empty(shape, like.options().dtype(dtype));
    given(*t, name, dtype, shape, like.device());
    return *t;
}

// A list from Python of as many tensors as the call takes: its elements are
// read by their place.
template <class T>
void count(const std::vector<T>& v, size_t n, const char* what)
{
    TORCH_CHECK_VALUE(v.size() == n, what, ", got ", v.size(), " tensors instead of ", n);
}

// bf16 or fp32 values; the ABI's dtype code
int32_t values(const Tensor& t, const char* name)
{
    TORCH_CHECK_TYPE(t.defined() && t.is_cuda(), name, " must be a CUDA (HIP) tensor");
    TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat, name,
                     " must be torch.bfloat16 or torch.float32, got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    return t.scalar_type() == at::kFloat ? MHC_FP32 : MHC_BF16;
}

at::ScalarType type_of(int32_t dtype) { return dtype == MHC_FP32 ? at::kFloat : at::kBFloat16; }

std::vector<int64_t> scale_shape(at::IntArrayRef shape)
{
    std::vector<int64_t> s(shape.begin(), shape.end());
    s.back() = (s.back() + kBlock - 1) / kBlock;
    return s;
}

void* stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

const float* f32(const Tensor& t) { return static_cast<const float*>(t.const_data_ptr()); }
const uint8_t* u8(const Tensor& t) { return static_cast<const uint8_t*>(t.const_data_ptr()); }
float* f32_out(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }
uint8_t* u8_out(const Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

struct Shape3 {
    int64_t T, n, C;
};

Shape3 streams(const Tensor& x, const char* name)
{
    need(x, name, at::kBFloat16);
    TORCH_CHECK_VALUE(x.dim() == 3, name, " must be [T, n, C]");
    return Shape3{x.size(0), x.size(1), x.size(2)};
}

// Solver options as (solver, max_iters, tol, warm_sweeps); negative tol = default.
mhc_proj_opts solver_opts(int32_t solver, int32_t max_iters, double tol, int32_t warm_sweeps)
{
    mhc_proj_opts o;
    mhc_proj_opts_default(&o);
    o.solver = solver;
    o.max_iters = max_iters;
    if (tol >= 0) o.tol = (float)tol;
    o.warm_sweeps = warm_sweeps;
    return o;
}

using Opts = std::tuple<int32_t, int32_t, double, int32_t>;

mhc_proj_opts solver_opts(const Opts& o)
{
    return solver_opts(std::get<0>(o), std::get<1>(o), std::get<2>(o), std::get<3>(o));
}

// ---------------------------------------------------------------------------
// checkpoints
// ---------------------------------------------------------------------------

std::tuple<int, Tensor, Tensor> ckpt_pack(const Tensor& x, int32_t format, const Opt& codes_out,
                                          const Opt& scales_out)
{
    const int32_t dt = values(x, "x");
    TORCH_CHECK_VALUE(x.dim() >= 1, "x must be [..., C]");
    const int64_t C = x.size(-1);
    const c10::DeviceGuard guard(x.device());
    Tensor codes = output(codes_out, "out codes", at::kByte, x.sizes(), x);
    Tensor scales = output(scales_out, "out scales", at::kByte, scale_shape(x.sizes()), x);
    const int st = mhc_ckpt_pack(x.const_data_ptr(), dt, codes.data_ptr(), u8_out(scales),
                                 C ? x.numel() / C : 0, C, format, stream_of(x));
    return {st, std::move(codes), std::move(scales)};
}

std::tuple<int, Tensor> ckpt_unpack(const Tensor& codes, const Tensor& scales, int32_t format,
                                    int32_t dtype, const Opt& out)
{
    need(codes, "codes", at::kByte);
    TORCH_CHECK_VALUE(codes.dim() >= 1, "codes must be [..., C]");
    given(scales, "scales", at::kByte, scale_shape(codes.sizes()), codes.device());
    const int64_t C = codes.size(-1);
    const c10::DeviceGuard guard(codes.device());
    Tensor x = output(out, "out", type_of(dtype), codes.sizes(), codes);
    const int st = mhc_ckpt_unpack(codes.const_data_ptr(), u8(scales), x.data_ptr(), dtype,
                                   C ? codes.numel() / C : 0, C, format, stream_of(codes));
    return {st, std::move(x)};
}

// src: H, or logits to be projected if opts is given
std::tuple<int, Tensor, Opt, Tensor, Tensor> stream_mix_ckpt(
    const Tensor& x, const Tensor& src, int32_t format, const c10::optional<Opts>& opts, bool return_H,
    const Opt& out, const Opt& H_out, const Opt& codes_out, const Opt& scales_out)
{
    const Shape3 s = streams(x, "x");
    given(src, opts ? "logits" : "H", at::kFloat, {s.T, s.n, s.n}, x.device());
    const c10::DeviceGuard guard(x.device());
    Tensor y = output(out, "out", at::kBFloat16, x.sizes(), x);
    Opt H;
    if (opts && return_H) H = output(H_out, "H_out", at::kFloat, src.sizes(), x);
    Tensor codes = output(codes_out, "ckpt codes", at::kByte, x.sizes(), x);
    Tensor scales = output(scales_out, "ckpt scales", at::kByte, scale_shape(x.sizes()), x);
    mhc_proj_opts o;
    if (opts) o = solver_opts(*opts);
    const int st = mhc_stream_mix_ckpt(x.const_data_ptr(), f32(src), H ? f32_out(*H) : nullptr,
                                       y.data_ptr(), codes.data_ptr(), u8_out(scales), s.T,
                                       (int32_t)s.n, s.C, format, opts ? &o : nullptr, stream_of(x));
    return {st, std::move(y), std::move(H), std::move(codes), std::move(scales)};
}

std::tuple<int, Tensor, Tensor> stream_mix_bwd_ckpt(const Tensor& codes, const Tensor& scales,
                                                    const Tensor& H, const Tensor& grad_out,
                                                    int32_t format, const Opt& gx_out,
                                                    const Opt& gH_out)
{
    const Shape3 s = streams(grad_out, "grad_out");
    given(codes, "ckpt codes", at::kByte, grad_out.sizes(), grad_out.device());
    given(scales, "ckpt scales", at::kByte, scale_shape(grad_out.sizes()), grad_out.device());
    given(H, "H", at::kFloat, {s.T, s.n, s.n}, grad_out.device());
    const c10::DeviceGuard guard(grad_out.device());
    Tensor gx = output(gx_out, "grad_x", at::kBFloat16, grad_out.sizes(), grad_out);
    Tensor gH = output(gH_out, "grad_H", at::kFloat, H.sizes(), grad_out);
    const int st = mhc_stream_mix_bwd_ckpt(codes.const_data_ptr(), u8(scales), f32(H),
                                           grad_out.const_data_ptr(), gx.data_ptr(), f32_out(gH), s.T,
                                           (int32_t)s.n, s.C, format, stream_of(grad_out));
    return {st, std::move(gx), std::move(gH)};
}

// The per-token maps of the layer step, in the order rms, logits, H_pre,
// H_post, H_res.
const char* const kMapNames[5] = {"rms", "logits", "H_pre", "H_post", "H_res"};

std::vector<int64_t> map_shape(int k, int64_t T, int64_t n)
{
    switch (k) {
    case 0: return {T};
    case 1: return {T, n * n + 2 * n};
    case 4: return {T, n, n};
    default: return {T, n};
    }
}

void set_maps(mhc_layer_args& a, const std::vector<Tensor>& m)
{
    a.rms = f32_out(m[0]);
    a.logits = f32_out(m[1]);
    a.H_pre = f32_out(m[2]);
    a.H_post = f32_out(m[3]);
    a.H_res = f32_out(m[4]);
}

std::vector<Tensor> new_maps(const std::vector<Opt>& out, const Shape3& s, const Tensor& like)
{
    std::vector<Tensor> m(5);
    for (int k = 0; k < 5; ++k)
        m[k] = output(out.empty() ? Opt() : out[k], kMapNames[k], at::kFloat, map_shape(k, s.T, s.n), like);
    return m;
}

void given_W(const Tensor& W, const Shape3& s, const at::Device& device)
{
    given(W, "W", at::kBFloat16, {s.n * s.n + 2 * s.n, s.n * s.C}, device);
}

mhc_layer_args layer_args(const Shape3& s, double eps, const mhc_proj_opts* opts)
{
    mhc_layer_args a{};
    a.T = s.T;
    a.n = (int32_t)s.n;
    a.C = s.C;
    a.eps = (float)eps;
    a.proj = opts;
    return a;
}

// The workspace of the maps, if the shape needs one, set in a.
Tensor read_workspace(mhc_layer_args& a, const Tensor& like)
{
    Tensor ws;
    const int64_t n = mhc_layer_read_workspace_bytes(a.T, a.n, a.C);
    if (n > 0) {
        ws = at::empty({n}, like.options().dtype(at::kByte));
        a.workspace = ws.data_ptr();
        a.workspace_bytes = n;
    }
    return ws;
}

// maps_out: empty or 5 optional buffers; outs: u, x_out; ckpt: x codes, x
// scales, f codes, f scales.
std::tuple<int, std::vector<Tensor>, std::vector<Tensor>, std::vector<Tensor>> layer_fwd_ckpt(
    const Tensor& x, const Tensor& W, const Tensor& f, int32_t format, double eps, const Opts& opts,
    const std::vector<Opt>& maps_out, const std::vector<Opt>& outs, const std::vector<Opt>& ckpt)
{
    if (!maps_out.empty()) count(maps_out, 5, "out must hold the 5 maps");
    count(outs, 2, "out must hold u and x_out");
    count(ckpt, 4, "ckpt must hold (codes, scales) of x and of f");
    const Shape3 s = streams(x, "x");
    given_W(W, s, x.device());
    given(f, "f", at::kBFloat16, {s.T, s.C}, x.device());
    const c10::DeviceGuard guard(x.device());
    std::vector<Tensor> maps = new_maps(maps_out, s, x);
    std::vector<Tensor> o{output(outs[0], "u", at::kBFloat16, {s.T, s.C}, x),
                          output(outs[1], "x_out", at::kBFloat16, x.sizes(), x)};
    std::vector<Tensor> c{output(ckpt[0], "ckpt x codes", at::kByte, x.sizes(), x),
                          output(ckpt[1], "ckpt x scales", at::kByte, scale_shape(x.sizes()), x),
                          output(ckpt[2], "ckpt f codes", at::kByte, f.sizes(), x),
                          output(ckpt[3], "ckpt f scales", at::kByte, scale_shape(f.sizes()), x)};
    const mhc_proj_opts po = solver_opts(opts);
    mhc_layer_args a = layer_args(s, eps, &po);
    a.x = x.const_data_ptr();
    a.W = W.const_data_ptr();
    a.f = f.const_data_ptr();
    a.u = o[0].data_ptr();
    a.x_out = o[1].data_ptr();
    set_maps(a, maps);
    const Tensor ws = read_workspace(a, x);
    const mhc_layer_ckpt k{format, c[0].data_ptr(), u8_out(c[1]), c[2].data_ptr(), u8_out(c[3])};
    const int st = mhc_layer_fwd_ckpt(&a, &k, stream_of(x));
    return {st, std::move(maps), std::move(o), std::move(c)};
}

// maps: the forward's 5; outs: optional grad_x, grad_f, grad_W, grad_logits.
std::tuple<int, std::vector<Tensor>> layer_bwd_ckpt(
    const std::vector<Tensor>& ckpt, const Tensor& W, const std::vector<Tensor>& maps,
    const Tensor& grad_x_out, const Tensor& grad_u, int32_t format, const Opt& workspace,
    const std::vector<Opt>& outs)
{
    count(ckpt, 4, "ckpt must hold (codes, scales) of x and of f");
    count(maps, 5, "fwd must hold the 5 maps");
    count(outs, 4, "out must hold the 4 gradients");
    const Shape3 s = streams(grad_x_out, "grad_x_out");
    const at::Device dev = grad_x_out.device();
    const std::vector<int64_t> fs{s.T, s.C};
    given(grad_u, "grad_u", at::kBFloat16, fs, dev);
    given_W(W, s, dev);
    given(ckpt[0], "ckpt x codes", at::kByte, grad_x_out.sizes(), dev);
    given(ckpt[1], "ckpt x scales", at::kByte, scale_shape(grad_x_out.sizes()), dev);
    given(ckpt[2], "ckpt f codes", at::kByte, fs, dev);
    given(ckpt[3], "ckpt f scales", at::kByte, scale_shape(fs), dev);
    for (int k = 0; k < 5; ++k) given(maps[k], kMapNames[k], at::kFloat, map_shape(k, s.T, s.n), dev);
    const c10::DeviceGuard guard(dev);
    const int64_t maps24 = s.n * s.n + 2 * s.n;
    std::vector<Tensor> o{output(outs[0], "grad_x", at::kBFloat16, grad_x_out.sizes(), grad_x_out),
                          output(outs[1], "grad_f", at::kBFloat16, fs, grad_x_out),
                          output(outs[2], "grad_W", at::kFloat, {maps24, s.n * s.C}, grad_x_out),
                          output(outs[3], "grad_logits", at::kFloat, {s.T, maps24}, grad_x_out)};
    Tensor ws;
    if (workspace.has_value()) {
        need(*workspace, "workspace", at::kByte);
        TORCH_CHECK_VALUE(workspace->device() == dev, "workspace must be on ", dev, ", got ",
                          workspace->device());
        ws = *workspace;
    } else {
        const int64_t n = mhc_layer_ckpt_workspace_bytes(s.T, (int32_t)s.n, s.C);
        ws = at::empty({n > 1 ? n : 1}, grad_x_out.options().dtype(at::kByte));
    }
    mhc_layer_args a = layer_args(s, 1e-6, nullptr);
    a.W = W.const_data_ptr();
    set_maps(a, maps);
    a.grad_x_out = grad_x_out.const_data_ptr();
    a.grad_u = grad_u.const_data_ptr();
    a.grad_x = o[0].data_ptr();
    a.grad_f = o[1].data_ptr();
    a.grad_W = f32_out(o[2]);
    a.grad_logits = f32_out(o[3]);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = ws.numel();
    const mhc_layer_ckpt k{format, ckpt[0].data_ptr(), u8_out(ckpt[1]), ckpt[2].data_ptr(), u8_out(ckpt[3])};
    const int st = mhc_layer_bwd_ckpt(&a, &k, stream_of(grad_x_out));
    return {st, std::move(o)};
}

// u4: the quantised u is wanted; keep_u: the bf16 u is.  Returns the maps, then
// u (if kept), codes, scales (if quantised).
std::tuple<int, std::vector<Tensor>, Opt, Opt, Opt> layer_read(
    const Tensor& x, const Tensor& W, bool u4, bool keep_u, double eps, const Opts& opts,
    const std::vector<Opt>& maps_out, const Opt& u_out, const Opt& codes_out, const Opt& scales_out)
{
    if (!maps_out.empty()) count(maps_out, 5, "out must hold the 5 maps");
    const Shape3 s = streams(x, "x");
    given_W(W, s, x.device());
    TORCH_CHECK_VALUE(s.C % 2 == 0, "C must be even");
    const c10::DeviceGuard guard(x.device());
    std::vector<Tensor> maps = new_maps(maps_out, s, x);
    Opt u, codes, scales;
    if (keep_u) u = output(u_out, "u", at::kBFloat16, {s.T, s.C}, x);
    if (u4) {
        codes = output(codes_out, "u codes", at::kByte, {s.T, s.C / 2}, x);
        scales = output(scales_out, "u scales", at::kByte, {s.T, s.C / kBlock}, x);
    }
    const mhc_proj_opts po = solver_opts(opts);
    mhc_layer_args a = layer_args(s, eps, &po);
    a.x = x.const_data_ptr();
    a.W = W.const_data_ptr();
    a.u = u ? u->data_ptr() : nullptr;
    set_maps(a, maps);
    const Tensor ws = read_workspace(a, x);
    const int st = mhc_layer_read(&a, codes ? codes->data_ptr() : nullptr, scales ? u8_out(*scales) : nullptr,
                                  stream_of(x));
    return {st, std::move(maps), std::move(u), std::move(codes), std::move(scales)};
}

// ---------------------------------------------------------------------------
// 4 bits
// ---------------------------------------------------------------------------

std::tuple<int, Tensor, Tensor> mx4_quantize(const Tensor& x, bool transpose, const Opt& codes_out,
                                             const Opt& scales_out)
{
    const int32_t dt = values(x, "x");
    TORCH_CHECK_VALUE(x.dim() == 2, "x must be [R, C]");
    const int64_t R = x.size(0), C = x.size(1);
    const int64_t rows = transpose ? C : R, cols = transpose ? R : C;
    TORCH_CHECK_VALUE(cols % kBlock == 0, "the quantised axis must be a multiple of ", kBlock, ", got ", cols);
    const c10::DeviceGuard guard(x.device());
    Tensor codes = output(codes_out, "codes", at::kByte, {rows, cols / 2}, x);
    Tensor scales = output(scales_out, "scales", at::kByte, {rows, cols / kBlock}, x);
    const int st = mhc_mx4_quantize(x.const_data_ptr(), dt, codes.data_ptr(), u8_out(scales), R, C,
                                    transpose ? 1 : 0, stream_of(x));
    return {st, std::move(codes), std::move(scales)};
}

// [R, C] values to be packed along rows and columns alike
void square_blocks(const Tensor& x, const char* name)
{
    TORCH_CHECK_VALUE(x.dim() == 2 && x.size(0) % kBlock == 0 && x.size(1) % kBlock == 0, name,
                      " must be [R, C] with R and C multiples of ", kBlock, ", got ", x.sizes());
}

struct Pair {
    Tensor codes, scales;
};

// a new 4-bit [R, C] matrix
Pair new_mx4(const Tensor& like, int64_t R, int64_t C)
{
    const auto o = like.options().dtype(at::kByte);
    return Pair{at::empty({R, C / 2}, o), at::empty({R, C / kBlock}, o)};
}

// codes, scales, transposed codes, transposed scales
std::tuple<int, Tensor, Tensor, Tensor, Tensor> mx4_quantize_both(const Tensor& x)
{
    const int32_t dt = values(x, "x");
    square_blocks(x, "x");
    const int64_t R = x.size(0), C = x.size(1);
    const c10::DeviceGuard guard(x.device());
    Pair r = new_mx4(x, R, C), t = new_mx4(x, C, R);
    const int st = mhc_mx4_quantize_both(x.const_data_ptr(), dt, r.codes.data_ptr(), u8_out(r.scales),
                                         t.codes.data_ptr(), u8_out(t.scales), R, C, stream_of(x));
    return {st, std::move(r.codes), std::move(r.scales), std::move(t.codes), std::move(t.scales)};
}

// codes, scales, checkpoint codes, checkpoint scales
std::tuple<int, Tensor, Tensor, Tensor, Tensor> mx4_quantize_ckpt(const Tensor& x, int32_t format)
{
    const int32_t dt = values(x, "x");
    TORCH_CHECK_VALUE(x.dim() == 2 && x.size(1) % kBlock == 0, "x must be [R, C] with C a multiple of ", kBlock,
                      ", got ", x.sizes());
    const int64_t R = x.size(0), C = x.size(1);
    const c10::DeviceGuard guard(x.device());
    Pair q = new_mx4(x, R, C);
    Tensor codes = at::empty(x.sizes(), x.options().dtype(at::kByte));
    Tensor scales = at::empty({R, C / kBlock}, x.options().dtype(at::kByte));
    const int st = mhc_mx4_quantize_ckpt(x.const_data_ptr(), dt, q.codes.data_ptr(), u8_out(q.scales),
                                         codes.data_ptr(), u8_out(scales), R, C, format, stream_of(x));
    return {st, std::move(q.codes), std::move(q.scales), std::move(codes), std::move(scales)};
}

std::tuple<int, Tensor, Tensor> mx4_requantize(const Tensor& codes, const Tensor& scales, int32_t format)
{
    need(codes, "codes", at::kByte);
    square_blocks(codes, "codes");
    const int64_t R = codes.size(0), C = codes.size(1);
    given(scales, "scales", at::kByte, {R, C / kBlock}, codes.device());
    const c10::DeviceGuard guard(codes.device());
    Pair t = new_mx4(codes, C, R);
    const int st = mhc_mx4_requantize(codes.const_data_ptr(), u8(scales), t.codes.data_ptr(), u8_out(t.scales), R,
                                      C, format, stream_of(codes));
    return {st, std::move(t.codes), std::move(t.scales)};
}

struct Mx4 {
    const void* codes;
    const uint8_t* scales;
    int64_t R, C;
};

Mx4 mx4(const Tensor& codes, const Tensor& scales, const char* name)
{
    need(codes, name, at::kByte);
    TORCH_CHECK_VALUE(codes.dim() == 2 && codes.size(1) % (kBlock / 2) == 0, name,
                      " codes must be [R, C/2] with C a multiple of ", kBlock);
    const int64_t R = codes.size(0), C = 2 * codes.size(1);
    given(scales, name, at::kByte, {R, C / kBlock}, codes.device());
    return Mx4{codes.const_data_ptr(), u8(scales), R, C};
}

std::tuple<int, Tensor> mx4_dequantize(const Tensor& codes, const Tensor& scales, int32_t dtype, const Opt& out)
{
    const Mx4 q = mx4(codes, scales, "quantised");
    const c10::DeviceGuard guard(codes.device());
    Tensor x = output(out, "out", type_of(dtype), {q.R, q.C}, codes);
    const int st = mhc_mx4_dequantize(q.codes, q.scales, x.data_ptr(), dtype, q.R, q.C, stream_of(codes));
    return {st, std::move(x)};
}

std::tuple<int, Tensor> mx4_matmul(const Tensor& ac, const Tensor& as, const Tensor& bc, const Tensor& bs,
                                   int32_t dtype, const Opt& out)
{
    const Mx4 a = mx4(ac, as, "a"), b = mx4(bc, bs, "b");
    TORCH_CHECK_VALUE(a.C == b.C && ac.device() == bc.device(), "a must be [M, ", b.C, "] on ", bc.device(),
                      ", got [", a.R, ", ", a.C, "] on ", ac.device());
    const c10::DeviceGuard guard(bc.device());
    Tensor y = output(out, "out", type_of(dtype), {a.R, b.R}, bc);
    const int st = mhc_mx4_matmul(a.codes, a.scales, b.codes, b.scales, y.data_ptr(), dtype, a.R, b.R, b.C,
                                  stream_of(bc));
    return {st, std::move(y)};
}

std::tuple<int, Tensor> mx4_matmul_values(const Tensor& a, const Tensor& bc, const Tensor& bs, int32_t dtype,
                                          const Opt& out)
{
    const int32_t ad = values(a, "a");
    const Mx4 b = mx4(bc, bs, "b");
    TORCH_CHECK_VALUE(a.dim() == 2 && a.size(1) == b.C && a.device() == bc.device(), "a must be [M, ", b.C,
                      "] on ", bc.device(), ", got ", a.sizes(), " on ", a.device());
    const int64_t M = a.size(0);
    const c10::DeviceGuard guard(bc.device());
    Tensor y = output(out, "out", type_of(dtype), {M, b.R}, bc);
    const int64_t n = mhc_mx4_matmul_values_workspace_bytes(M, b.R, b.C);
    Tensor ws;
    if (n > 0) ws = at::empty({n}, bc.options());
    const int st = mhc_mx4_matmul_values(a.const_data_ptr(), ad, b.codes, b.scales, y.data_ptr(), dtype, M, b.R,
                                         b.C, n > 0 ? ws.data_ptr() : nullptr, n > 0 ? n : 0, stream_of(bc));
    return {st, std::move(y)};
}

std::tuple<int, Tensor> mx4_write_back(const Tensor& ac, const Tensor& as, const Tensor& bc, const Tensor& bs,
                                       const Tensor& x, const Tensor& H_post, const Tensor& H_res,
                                       const Opt& out, const Opt& f_out)
{
    const Shape3 s = streams(x, "x");
    const Mx4 a = mx4(ac, as, "a"), b = mx4(bc, bs, "b");
    TORCH_CHECK_VALUE(a.R == s.T && b.R == s.C && a.C == b.C && ac.device() == x.device() &&
                          bc.device() == x.device(),
                      "a and b must be [", s.T, ", K] and [", s.C, ", K] on ", x.device(), ", got [", a.R, ", ",
                      a.C, "] on ", ac.device(), " and [", b.R, ", ", b.C, "] on ", bc.device());
    given(H_post, "H_post", at::kFloat, {s.T, s.n}, x.device());
    given(H_res, "H_res", at::kFloat, {s.T, s.n, s.n}, x.device());
    const c10::DeviceGuard guard(x.device());
    Tensor y = output(out, "out", at::kBFloat16, x.sizes(), x);
    if (f_out.has_value()) given(*f_out, "f_out", at::kBFloat16, {s.T, s.C}, x.device());
    const int st = mhc_mx4_write_back(a.codes, a.scales, b.codes, b.scales, x.const_data_ptr(), f32(H_post),
                                      f32(H_res), y.data_ptr(), f_out ? f_out->data_ptr() : nullptr, s.T,
                                      (int32_t)s.n, s.C, a.C, stream_of(x));
    return {st, std::move(y)};
}

// Inside a backward that is being captured: does a gradient go on, at once or
// through nodes in between (a leaf's cast or view), to a node whose stream is
// the default one, that is, to a graph begun eagerly?  The engine would make
// that stream wait for the capture, which HIP refuses, and the process ends on
// it; so the node before it raises instead.  An eager graph begun on another
// stream joins the capture and is no such case.  Nodes that this backward does
// not run are passed over.
bool leaves_capture()
{
    const auto node = torch::autograd::get_current_node();
    if (node == nullptr || c10::hip::currentStreamCaptureStatusMayInitCtx() != c10::hip::CaptureStatus::Active)
        return false;
    std::vector<torch::autograd::Node*> todo{node.get()};
    std::unordered_set<torch::autograd::Node*> seen{node.get()};
    while (!todo.empty()) {
        torch::autograd::Node* n = todo.back();
        todo.pop_back();
        for (size_t i = 0; i < n->num_outputs(); ++i) {
            torch::autograd::Node* next = n->next_edge(i).function.get();
            if (next == nullptr || !n->task_should_compute_output(i) || !seen.insert(next).second) continue;
            const auto stream = next->stream();
            if (stream.has_value() && stream->id() == 0) return true;
            todo.push_back(next);
        }
    }
    return false;
}

void stays_in_capture()
{
    TORCH_CHECK(!leaves_capture(),
                "a captured backward reaches an eager graph on the default stream: drop what holds that graph, or "
                "capture with leaves of its own");
}

void checked(int st)
{
    TORCH_CHECK(st == MHC_OK, "mhc: ", mhc_last_error());
}

// y = q(x) q(w)^T; grad_x = q(gy) q(w^T)^T and grad_w = q(gy^T) q(xhat^T)^T, with
// x kept as the checkpoint xhat.  A node of its own, so that the backward runs
// on autograd's thread without Python.
struct Mx4Linear : torch::autograd::Function<Mx4Linear> {
    static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& x0, const Tensor& w0,
                          int64_t format)
    {
        const Tensor x = x0.contiguous(), w = w0.contiguous();
        auto [sx, xc, xs, codes, scales] = mx4_quantize_ckpt(x, (int32_t)format);
        checked(sx);
        auto [sw, wc, ws] = mx4_quantize(w, false, Opt(), Opt());
        checked(sw);
        auto [sy, y] = mx4_matmul(xc, xs, wc, ws, values(x, "x"), Opt());
        checked(sy);
        ctx->save_for_backward({codes, scales, w});
        ctx->saved_data["format"] = format;
        return y;
    }

    static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                   torch::autograd::variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Tensor &codes = saved[0], &scales = saved[1], &w = saved[2];
        const int32_t format = (int32_t)ctx->saved_data["format"].toInt();
        const bool want_x = ctx->needs_input_grad(0), want_w = ctx->needs_input_grad(1);
        const bool twice = at::GradMode::is_enabled();
        const at::AutoGradMode no_grad(false);
        stays_in_capture();
        if (!grads[0].defined()) return {Tensor(), Tensor(), Tensor()};
        const Tensor gy = grads[0].contiguous();
        Tensor gx, gw;
        if (gy.size(0) == 0) {
            if (want_x) gx = at::zeros(codes.sizes(), gy.options());
            if (want_w) gw = at::zeros_like(w);
        } else {
            Pair r, t;
            int st = MHC_OK;
            if (want_x && want_w)
                std::tie(st, r.codes, r.scales, t.codes, t.scales) = mx4_quantize_both(gy);
            else if (want_x)
                std::tie(st, r.codes, r.scales) = mx4_quantize(gy, false, Opt(), Opt());
            else if (want_w)
                std::tie(st, t.codes, t.scales) = mx4_quantize(gy, true, Opt(), Opt());
            checked(st);
            if (want_x) {
                auto [sw, wc, ws] = mx4_quantize(w, true, Opt(), Opt());
                checked(sw);
                std::tie(st, gx) = mx4_matmul(r.codes, r.scales, wc, ws, values(gy, "grad"), Opt());
                checked(st);
            }
            if (want_w) {
                auto [sx, xc, xs] = mx4_requantize(codes, scales, format);
                checked(sx);
                std::tie(st, gw) = mx4_matmul(t.codes, t.scales, xc, xs, values(w, "w"), Opt());
                checked(st);
            }
        }
        if (!twice) return {gx, gw, Tensor()};
        // create_graph: a second derivative raises instead of being zero
        torch::autograd::variable_list out{gx, gw};
        for (Tensor& g : out)
            if (g.defined()) {
                const auto error = std::make_shared<torch::autograd::DelayedError>(
                    "mx4_linear is differentiable once", 1);
                g = (*error)({g.detach().set_requires_grad(true)})[0];
            }
        return {out[0], out[1], Tensor()};
    }
};

Tensor mx4_linear(const Tensor& x, const Tensor& w, int32_t format)
{
    return Mx4Linear::apply(x, w, (int64_t)format);
}

}  // namespace

PYBIND11_MODULE(_binding, m)
{
    m.def("ckpt_pack", &ckpt_pack);
    m.def("ckpt_unpack", &ckpt_unpack);
    m.def("stream_mix_ckpt", &stream_mix_ckpt);
    m.def("stream_mix_bwd_ckpt", &stream_mix_bwd_ckpt);
    m.def("layer_fwd_ckpt", &layer_fwd_ckpt);
    m.def("layer_bwd_ckpt", &layer_bwd_ckpt);
    m.def("layer_read", &layer_read);
    m.def("mx4_quantize", &mx4_quantize);
    m.def("mx4_quantize_both", &mx4_quantize_both);
    m.def("mx4_quantize_ckpt", &mx4_quantize_ckpt);
    m.def("mx4_requantize", &mx4_requantize);
    m.def("mx4_dequantize", &mx4_dequantize);
    m.def("mx4_matmul", &mx4_matmul);
    m.def("mx4_matmul_values", &mx4_matmul_values);
    m.def("mx4_write_back", &mx4_write_back);
    m.def("mx4_linear", &mx4_linear);
    m.def("stays_in_capture", &stays_in_capture);
}
