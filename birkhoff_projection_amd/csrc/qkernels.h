// Launchers of the checkpoint and 4-bit kernels behind the C ABI (internal;
// see include/mhc.h for the public contract).  Each returns
// hipGetLastError() after enqueueing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace mhc {

// Workgroups of the passes that take tokens b, b + G, ... (at most 16 each): 16
// tokens per workgroup, fewer where that would leave most of the chip idle.
inline unsigned token_grid(int64_t T)
{
    const int64_t full = (T + 15) / 16, most = T < 1024 ? T : 1024;
    return (unsigned)(full > most ? full : most);
}

// A packed tensor: codes and one scale byte per block of 32 columns of a row.
struct Packed {
    void* codes;
    uint8_t* scales;
};

// fmt: MxFormat (kE4M3, kInt8); f32: the values are fp32 instead of bf16.
hipError_t launch_ckpt_pack(const void* x, bool f32, const Packed& out, int64_t R, int64_t C,
                            int fmt, hipStream_t stream);
hipError_t launch_ckpt_unpack(const Packed& in, void* x, bool f32, int64_t R, int64_t C, int fmt,
                              hipStream_t stream);
hipError_t launch_stream_mix_ckpt(const void* x, const float* Hl, float* H_out, void* out,
                                  const Packed& ckpt, int64_t T, int64_t C, int fmt,
                                  const SolverOpts* proj, hipStream_t stream);
hipError_t launch_stream_mix_bwd_ckpt(const Packed& ckpt, const float* H, const void* gout,
                                      void* gx, float* gH, int64_t T, int64_t C, int fmt,
                                      hipStream_t stream);
hipError_t launch_mx4_quantize(const void* x, bool f32, const Packed& out, int64_t R, int64_t C,
                               bool transpose, hipStream_t stream);
// rows and, transposed, columns of x in one pass
hipError_t launch_mx4_quantize_both(const void* x, bool f32, const Packed& rows, const Packed& cols,
                                    int64_t R, int64_t C, hipStream_t stream);
// rows of x in 4 bits and as an 8-bit checkpoint in one pass
hipError_t launch_mx4_quantize_ckpt(const void* x, bool f32, const Packed& out, const Packed& ckpt,
                                    int64_t R, int64_t C, int fmt, hipStream_t stream);
// the columns of an 8-bit checkpoint [R, C] in 4 bits
hipError_t launch_mx4_requantize(const Packed& ckpt, const Packed& out, int64_t R, int64_t C, int fmt,
                                 hipStream_t stream);
hipError_t launch_mx4_dequantize(const Packed& in, void* x, bool f32, int64_t R, int64_t C,
                                 hipStream_t stream);
// y [M,N] = a b^T for MXFP4 a [M,K], b [N,K]; f32: y is fp32 instead of bf16.
hipError_t launch_mx4_matmul(const Packed& a, const Packed& b, void* out, bool f32, int64_t M,
                             int64_t N, int64_t K, hipStream_t stream);
// The same with a given as bf16 or fp32 values and quantised in the product's
// own kernel, for the shapes that mx4_fuses_quantize admits (few rows).
bool mx4_fuses_quantize(int64_t M, int64_t K);
hipError_t launch_mx4_matmul_fused(const void* a, bool a_f32, const Packed& b, void* out, bool f32,
                                   int64_t M, int64_t N, int64_t K, hipStream_t stream);
// x_out [T,4,C] = H_post (x) (a b^T) + H_res x, and a b^T itself to f_out if
// that is not NULL.
hipError_t launch_mx4_write_back(const Packed& a, const Packed& b, const void* x,
                                 const float* Hpost, const float* Hres, void* x_out, void* f_out,
                                 int64_t T, int64_t C, int64_t K, hipStream_t stream);

// The maps pass of the plain layer's forward (layer.hip), which the checkpointed
// step and the read half share.
hipError_t launch_layer_maps(const LayerPtrs& a, int64_t T, int64_t C, float eps,
                             const SolverOpts& o, hipStream_t stream);

// The read half of the layer step: a.rms .. a.H_res, and u as bf16 (a.u) and /
// or MXFP4 (u4), each if its pointer is not NULL.  a.workspace holds
// read_plan().bytes bytes (fp32 partials [splits][T][25]; none for many tokens).
struct ReadPlan {
    int64_t splits, steps_per, bytes;
    int tiles;  // of 16 tokens to a workgroup of the partial sums
};
ReadPlan read_plan(int64_t T, int64_t C);
// The partial sums of a plan that splits.
hipError_t launch_read_part(const LayerPtrs& a, const ReadPlan& p, int64_t T, int64_t C, hipStream_t stream);
hipError_t launch_layer_read(const LayerPtrs& a, const Packed& u4, int64_t T, int64_t C, float eps,
                             const SolverOpts& o, hipStream_t stream);

// Backward workspace: s[Tp] fp32 | dl / r in bf16 parts [Tp/32][3][24][32] |
// W^T [4C][24] bf16 | grad_W partials [groups][24][4C] fp32 (each 256-byte
// aligned).
struct LayerCkptPlan {
    int64_t Tp, group_tokens, groups;  // tokens padded to 64; groups of the grad_W pass
    int64_t off_s, off_dl, off_wt, off_partial;
    int64_t bytes;
};

LayerCkptPlan layer_ckpt_plan(int64_t T, int64_t C);

// The layer step with x and f kept as checkpoints (written by the forward,
// read by the backward in the place of a.x and a.f).
hipError_t launch_layer_fwd_ckpt(const LayerPtrs& a, const Packed& x, const Packed& f, int64_t T,
                                 int64_t C, float eps, int fmt, const SolverOpts& o,
                                 hipStream_t stream);
hipError_t launch_layer_bwd_ckpt(const LayerPtrs& a, const Packed& x, const Packed& f, int64_t T,
                                 int64_t C, int fmt, hipStream_t stream);

}  // namespace mhc
