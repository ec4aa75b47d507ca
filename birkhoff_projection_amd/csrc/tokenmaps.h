// A token's maps from the partial sums that read_part_kernel (read.hip) writes:
// shared by the kernels that finish a few tokens, one workgroup each.
#pragma once
#include "proj4.h"
#include "qkernels.h"

namespace mhc {

constexpr int kTokenMaps = 24;
constexpr int kTokenVals = kTokenMaps + 1;  // logits and the sum of squares

MHC_DEV float token_sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

struct TokenMaps {
    float* logits;
    float* rms;
    float* Hpre;
    float* Hpost;
    float* Hres;
};

struct TokenLds {
    float p[8][32];
    float l[kTokenVals];
};

// A workgroup of 256 sums token t's partials in a fixed order into s.l, and
// writes rms, logits, H_pre and H_post.  Returns 1 / rms.
MHC_DEV float token_logits(TokenLds& s, const float* __restrict__ partial, int splits, const TokenMaps& o,
                           int64_t t, int64_t T, int64_t C8, float eps)
{
    const int tid = threadIdx.x;
    {
        const int m = tid & 31, g = tid >> 5;
        float v = 0.f;
        if (m < kTokenVals)
            for (int k = g; k < splits; k += 8) v += partial[((int64_t)k * T + t) * kTokenVals + m];
        s.p[g][m] = v;
    }
    __syncthreads();
    if (tid < kTokenVals) {
        float v = 0.f;
#pragma unroll
        for (int g = 0; g < 8; ++g) v += s.p[g][tid];
        s.l[tid] = v;
    }
    __syncthreads();
    const float r = sqrtf(s.l[kTokenMaps] / (float)(32 * C8) + eps);
    const float inv = 1.f / r;
    if (tid < kTokenMaps) {
        const float l = s.l[tid] * inv;
        o.logits[kTokenMaps * t + tid] = l;
        if (tid == 0) o.rms[t] = r;
        if (tid < 4) o.Hpre[4 * t + tid] = token_sigmoid(l);
        else if (tid < 8) o.Hpost[4 * t + tid - 4] = token_sigmoid(l);
    }
    return inv;
}

// One lane projects the token's last 16 logits; h is H_res, written too.
template <int SOLVER>
MHC_DEV void token_project(const TokenLds& s, float inv, const TokenMaps& o, int64_t t, const SolverOpts& opts,
                           float* h)
{
    float a[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) a[k] = s.l[8 + k] * inv;
    if (SOLVER == 0)
        project_newton(a, h, opts);
    else
        project_sinkhorn(a, h, opts);
    float4* ho = reinterpret_cast<float4*>(o.Hres + 16 * t);
#pragma unroll
    for (int q = 0; q < 4; ++q) ho[q] = make_float4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
}

}  // namespace mhc
