// Launchers of the checkpoint and 4-bit kernels behind the C ABI (internal;
// see include/mhc.h for the public contract).  Each returns
// hipGetLastError() after enqueueing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace mhc {

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
hipError_t launch_mx4_dequantize(const Packed& in, void* x, bool f32, int64_t R, int64_t C,
                                 hipStream_t stream);

// Parts of the plain layer step (layer.hip) that the checkpointed one shares:
// the maps pass of the forward, the transposition of W to [4C][24] bf16, and
// the sum of the grad_W partials over the token groups.
hipError_t launch_layer_maps(const LayerPtrs& a, int64_t T, int64_t C, float eps,
                             const SolverOpts& o, hipStream_t stream);
hipError_t launch_layer_wt(const void* W, void* Wt, int64_t C, hipStream_t stream);
hipError_t launch_layer_dw_reduce(const float* partial, float* gW, int64_t C, int64_t groups,
                                  hipStream_t stream);

// Backward workspace: s[Tp] fp32 | dl^T / r in three bf16 parts [3][24][Tp] |
// W^T [4C][24] bf16 | grad_W partials [groups][24][4C] fp32 (each 256-byte
// aligned).
struct LayerCkptPlan {
    int64_t Tp, group_tokens, groups;  // as in LayerPlan
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
