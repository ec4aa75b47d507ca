// The residual-layer step (layer.hip) with x and f kept as 8-bit checkpoints
// (mxfmt.h) between forward and backward, for gfx950.
//
//   mix    read-mix and write-back, and x and f packed in the same pass
//   dots   per-token reductions from the checkpoints (read only); epilogue:
//          sigmoid derivative and projection backward -> grad_logits
//   dx     grad_x, grad_f
//   dw     grad_W partials on MFMA
// The maps of the forward come from the partial sums of the layer's read half
// (read.hip) or from the plain layer's maps pass, as there.
//
// The formulas are the plain layer's with xhat, fhat (what the checkpoints
// stand for) in the place of x, f; the forward's r, logits and maps are those
// of x itself.  Checkpoints are half the bytes of x in each of the three
// backward passes that read it.
//
// Mixed precision: a checkpoint value is exact in bf16, so MFMA takes it
// unrounded.  grad_logits / r enters the grad_W product as three bf16 parts,
// which hold all 24 bits of an fp32 (its sum over the tokens is then as good
// as in fp32), and the grad_x product as two, enough for a bf16 result.
#include "ldscopy.h"
#include "mxfmt.h"
#include "proj4.h"
#include "qkernels.h"
#include "tokenmaps.h"
#include "wave.h"

namespace mhc {

namespace {

constexpr int kBlock = 256;
constexpr int kMaps = 24;  // n*n + 2n for n = 4

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

MHC_DEV bf16x8 as_bf16x8(const uint4& q) { return __builtin_bit_cast(bf16x8, q); }

// Projection backward of one matrix (project_bwd in proj4.h), solved twice:
// the column sums of dA, which the exact solution makes zero, are the residual
// of the first solve, and a second solve takes them off.  The first carries
// the ridge's relative error of a few 1e-6, thirty times the rounding of its
// inputs; after the second 2e-7 is left (N(0,1) logits, G from C = 1024 wide
// dots).  Where a curvature lies below the ridge both solves damp it alike.
MHC_DEV void project_bwd_refined(const float* P, const float* G, float* dA)
{
    const Weights w = laplacian_weights(P);
    const float lam = ridge(w);
    float be[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int it = 0; it < 3; ++it) {
        float rhs[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float h[4] = {G[4 * i] - be[0], G[4 * i + 1] - be[1], G[4 * i + 2] - be[2], G[4 * i + 3]};
            float hc[4];
            centred_row(P + 4 * i, h, hc);
#pragma unroll
            for (int j = 0; j < 4; ++j) dA[4 * i + j] = P[4 * i + j] * hc[j];
#pragma unroll
            for (int j = 0; j < 3; ++j) rhs[j] += dA[4 * i + j];
        }
        if (it < 2) {
            float d0, d1, d2;
            laplacian_solve(w.w01, w.w02, w.w03, w.w12, w.w13, w.w23, lam, rhs[0], rhs[1], rhs[2],
                            d0, d1, d2);
            be[0] += d0;
            be[1] += d1;
            be[2] += d2;
        }
    }
}

// dl / r as an MFMA operand: bf16 parts of 32 tokens' maps,
// [T / 32][part][map][32 tokens].  The tokens of one product step lie
// together: one chunk is one run of bytes, and with whole rows of tokens per map
// 16384 tokens put every map of a step on the same L2 channel.
constexpr int kDlParts = 3;

MHC_DEV int64_t dl_at(int64_t t, int part, int map)
{
    return ((t >> 5) * kDlParts + part) * (kMaps * 32) + map * 32 + (t & 31);
}

// One chunk of 8 columns of token t: u, x_out and both checkpoints from the
// chunk of x and f.  Quads of lanes are whole (C8 is a multiple of 8).
template <int FMT>
MHC_DEV void layer_mix_chunk(const float (&M)[kMaps], const uint4 (&xq)[4], const uint4& fq, int64_t t, int64_t c,
                             int64_t C8, uint4* __restrict__ u, uint4* __restrict__ xo, uint2* __restrict__ xc,
                             uint8_t* __restrict__ xs_out, uint2* __restrict__ fc, uint8_t* __restrict__ fs_out)
{
    float xs[4][8], ff[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) mx_unpack8(xq[j], xs[j]);
    mx_unpack8(fq, ff);
    float uu[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float s = M[0] * xs[0][e];
        s = __builtin_fmaf(M[1], xs[1][e], s);
        s = __builtin_fmaf(M[2], xs[2][e], s);
        uu[e] = __builtin_fmaf(M[3], xs[3][e], s);
    }
    mhc_store_stream(&u[t * C8 + c], mx_pack8(uu));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float o8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float s = M[4 + i] * ff[e];
            s = __builtin_fmaf(M[8 + 4 * i + 0], xs[0][e], s);
            s = __builtin_fmaf(M[8 + 4 * i + 1], xs[1][e], s);
            s = __builtin_fmaf(M[8 + 4 * i + 2], xs[2][e], s);
            o8[e] = __builtin_fmaf(M[8 + 4 * i + 3], xs[3][e], s);
        }
        mhc_store_stream(&xo[(t * 4 + i) * C8 + c], mx_pack8(o8));
    }
    const bool lead = (c & 3) == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t m = mx_quad_max(mx_amax8(xq[j])), s = mx_scale_byte<FMT>(m);
        mx_store_stream(&xc[(t * 4 + j) * C8 + c], mx_encode8<FMT>(xs[j], m, s));
        if (lead) xs_out[(t * 4 + j) * (C8 / 4) + (c >> 2)] = (uint8_t)s;
    }
    const uint32_t m = mx_quad_max(mx_amax8(fq)), s = mx_scale_byte<FMT>(m);
    mx_store_stream(&fc[t * C8 + c], mx_encode8<FMT>(ff, m, s));
    if (lead) fs_out[t * (C8 / 4) + (c >> 2)] = (uint8_t)s;
}

// ---------------------------------------------------------------------------
// mix: read-mix u, write-back x_out and the checkpoints of x and f, 16 tokens
// per workgroup (spaced by the grid size, so the workgroups stream a
// contiguous front), 2^shift threads to a token.  Bound by memory: 16384 x 7168
// 541-549 us, 5.4 TB/s.
// ---------------------------------------------------------------------------
constexpr int kMixTokens = 16;

template <int FMT, bool NARROW>
__global__ __launch_bounds__(kBlock) void layer_mix_ckpt_kernel(
    const uint4* __restrict__ x, const uint4* __restrict__ f, const float* __restrict__ Hpre,
    const float* __restrict__ Hpost, const float* __restrict__ Hres, uint4* __restrict__ u,
    uint4* __restrict__ xo, uint2* __restrict__ xc, uint8_t* __restrict__ xs_out,
    uint2* __restrict__ fc, uint8_t* __restrict__ fs_out, int64_t T, int64_t C8,
    int shift)
{
    __shared__ float sM[kMixTokens][kMaps];
    const int64_t b = blockIdx.x, G = gridDim.x;
    const int tid = threadIdx.x;
    const int64_t per = (T - b + G - 1) / G;
    const int nt = (int)(per < kMixTokens ? per : kMixTokens);
    for (int p = tid; p < nt * kMaps; p += kBlock) {
        const int tl = p / kMaps, m = p % kMaps;
        const int64_t t = b + G * tl;
        sM[tl][m] = m < 4 ? Hpre[4 * t + m] : (m < 8 ? Hpost[4 * t + m - 4] : Hres[16 * t + m - 8]);
    }
    __syncthreads();
    for (int tl = first_token<NARROW>(tid, shift); tl < nt; tl += kBlock >> shift) {
        float M[kMaps];
#pragma unroll
        for (int m = 0; m < kMaps; ++m) M[m] = sM[tl][m];
        const int64_t t = b + G * tl;
        // C8 is a multiple of 8: a quad of lanes (one block) is whole
        for (int64_t c = tid & ((1 << shift) - 1); c < C8; c += 1 << shift) {
            uint4 xq[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) xq[j] = mhc_load_stream(&x[(t * 4 + j) * C8 + c]);
            const uint4 fq = mhc_load_stream(&f[t * C8 + c]);
            layer_mix_chunk<FMT>(M, xq, fq, t, c, C8, u, xo, xc, xs_out, fc, fs_out);
        }
    }
}

// Where the maps' sums are split (read.hip): a workgroup per token finishes its
// maps and goes on to the mix, whose first chunks of x and f are under way
// meanwhile (forward in a graph, us, against maps and mix one after the other:
// 1 x 7168 15 / 17, 300 x 256 12.5 / 15.3, 4096 x 7168 191 / 213).
template <int SOLVER, int FMT>
__global__ __launch_bounds__(kBlock) void layer_finish_ckpt_kernel(
    const uint4* __restrict__ x, const uint4* __restrict__ f, const float* __restrict__ partial, int splits,
    TokenMaps maps, uint4* __restrict__ u, uint4* __restrict__ xo, uint2* __restrict__ xc,
    uint8_t* __restrict__ xs_out, uint2* __restrict__ fc, uint8_t* __restrict__ fs_out, int64_t T, int64_t C8,
    float eps, SolverOpts opts)
{
    __shared__ TokenLds s;
    __shared__ float sM[kMaps];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    uint4 xq[4], fq;
    const auto load = [&](int64_t c) {
        c = c < C8 ? c : C8 - 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) xq[j] = mhc_load_stream(&x[(t * 4 + j) * C8 + c]);
        fq = mhc_load_stream(&f[t * C8 + c]);
    };
    load(tid);
    const float inv = token_logits(s, partial, splits, maps, t, T, C8, eps);
    if (tid < 8) sM[tid] = token_sigmoid(s.l[tid] * inv);
    if (tid == 64) token_project<SOLVER>(s, inv, maps, t, opts, &sM[8]);
    __syncthreads();
    float M[kMaps];
#pragma unroll
    for (int m = 0; m < kMaps; ++m) M[m] = sM[m];
    for (int64_t c = tid; c < C8; c += kBlock) {
        if (c != tid) load(c);
        layer_mix_chunk<FMT>(M, xq, fq, t, c, C8, u, xo, xc, xs_out, fc, fs_out);
    }
}

// ---------------------------------------------------------------------------
// dots: a wave handles tw consecutive tokens (up to 16, fewer where that
// would leave waves missing), one at a time across the wave; lanes stride over
// the 8-column chunks.  The (token, chunk) steps of a wave form one software
// pipeline: step i+1's loads are issued into the other register set before
// step i is consumed (the vector-memory counter retires in order), across
// token boundaries too.  At a token's last chunk the 24 partial dots are
// wave-reduced into LDS; then lanes 0..tw-1 each finish one token.  Narrow
// rows (W = 16): 16 lanes to a token, four tokens at a time.  Reads only, bound by
// memory: 16384 x 7168 311-315 us, 5.6 TB/s.
// ---------------------------------------------------------------------------
struct DotsLoads {
    uint2 x[4], f;
    uint32_t sx[4], sf;
    uint4 g[4], u;
};

struct DotsLane {
    const uint2* xc;
    const uint8_t* xs;
    const uint2* fc;
    const uint8_t* fs;
    const uint4* gxo;
    const uint4* gu;
    int64_t T, C8, tb;
    int nch, lane;  // chunks of W lanes in a row
};

// Place in a wave's sequence of steps: token tl, chunk ci of it.
struct DotsStep {
    int tl, ci;
};

MHC_DEV DotsStep dots_next(const DotsStep& s, int nch)
{
    const bool last = s.ci + 1 == nch;
    return DotsStep{last ? s.tl + 1 : s.tl, last ? 0 : s.ci + 1};
}

template <int W>
MHC_DEV int64_t dots_token(const DotsLane& L, const DotsStep& s)
{
    return W == 64 ? L.tb + s.tl : L.tb + (int64_t)(64 / W) * s.tl + L.lane / W;
}

template <int W>
MHC_DEV void dots_issue(const DotsLane& L, DotsLoads& d, const DotsStep& s)
{
    // steps past the wave's last one read clamped addresses and are never consumed
    int64_t t = dots_token<W>(L, s);
    t = t < L.T ? t : L.T - 1;
    int64_t c = (L.lane & (W - 1)) + W * (int64_t)s.ci;
    c = c < L.C8 ? c : L.C8 - 1;
    const int64_t cb = L.C8 / 4, b = c >> 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        d.x[j] = L.xc[(t * 4 + j) * L.C8 + c];
        d.sx[j] = L.xs[(t * 4 + j) * cb + b];
        d.g[j] = L.gxo[(t * 4 + j) * L.C8 + c];
    }
    d.f = L.fc[t * L.C8 + c];
    d.sf = L.fs[t * cb + b];
    d.u = L.gu[t * L.C8 + c];
}

template <int FMT, int W>
MHC_DEV void dots_consume(const DotsLane& L, const DotsLoads& d, const DotsStep& s, float (&acc)[32],
                          float (*sDots)[kMaps])
{
    const int64_t t = dots_token<W>(L, s);
    const int64_t c = (L.lane & (W - 1)) + W * (int64_t)s.ci;
    if (t < L.T && c < L.C8) {
        float sc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = mx_scale(d.sx[j]);
        const float sf = mx_scale(d.sf);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 4 columns at a time
            float xs[4][4], gs[4][4], ff[4], uu[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mx_decode4<FMT>(h ? d.x[j].y : d.x[j].x, sc[j], xs[j]);
                const uint32_t w0 = h ? d.g[j].z : d.g[j].x, w1 = h ? d.g[j].w : d.g[j].y;
                gs[j][0] = mhc_bf16_lo(w0);
                gs[j][1] = mhc_bf16_hi(w0);
                gs[j][2] = mhc_bf16_lo(w1);
                gs[j][3] = mhc_bf16_hi(w1);
            }
            mx_decode4<FMT>(h ? d.f.y : d.f.x, sf, ff);
            const uint32_t w0 = h ? d.u.z : d.u.x, w1 = h ? d.u.w : d.u.y;
            uu[0] = mhc_bf16_lo(w0);
            uu[1] = mhc_bf16_hi(w0);
            uu[2] = mhc_bf16_lo(w1);
            uu[3] = mhc_bf16_hi(w1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = __builtin_fmaf(uu[e], xs[j][e], acc[j]);
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[4 + k] = __builtin_fmaf(gs[k][e], ff[e], acc[4 + k]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[8 + 4 * k + j] = __builtin_fmaf(gs[k][e], xs[j][e], acc[8 + 4 * k + j]);
            }
        }
    }
    if (s.ci == L.nch - 1) {  // the token's last chunk: reduce its dots
        if (W == 64) {
            const float sm = wave_sum_halving<32>(acc);
            const int idx = (L.lane >> 1) & 31;
            if ((L.lane & 1) == 0 && idx < kMaps) sDots[s.tl][idx] = sm;
        } else {
            sum16_halving<32>(acc);
            const int idx = 2 * (L.lane & 15);
            if (idx < kMaps) {
                float* d = sDots[(64 / W) * s.tl + L.lane / W];
                d[idx] = acc[0];
                d[idx + 1] = acc[1];
            }
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[k] = 0.f;
    }
}

// What a token's dots become: sigmoid derivative, projection backward, the
// RMSNorm coefficient, and dl / r as the operand of the grad_W pass.
struct DotsOut {
    const float* Hpre;
    const float* Hpost;
    const float* Hres;
    const float* logits;
    const float* rms;
    float* glogits;
    float* svec;
    __bf16* dlT;
    int64_t T, D;  // tokens; D = 4C
};

// W [24, 4C] transposed, [4C][24], by the workgroups of a dots launch behind
// those of the tokens: one launch less (the pass over dx wants it next).
struct WtOut {
    const uint16_t* W;
    uint4* Wt;
    unsigned first;  // workgroup
};

MHC_DEV void transpose_W(const WtOut& o, int64_t D)
{
    const int64_t k = (int64_t)(blockIdx.x - o.first) * kBlock + threadIdx.x;
    if (k >= D) return;
    uint4 v[kMaps / 8];
    uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
    for (int m = 0; m < kMaps; m += 2) w[m / 2] = o.W[m * D + k] | (uint32_t)o.W[(m + 1) * D + k] << 16;
#pragma unroll
    for (int q = 0; q < kMaps / 8; ++q) o.Wt[kMaps / 8 * k + q] = v[q];
}

// One lane finishes token t (tokens from T on: zeros for the grad_W pass).
MHC_DEV void finish_token(const DotsOut& o, int64_t t, const float* dots)
{
    float dl[kMaps];
    if (t < o.T) {
        float d[kMaps];
#pragma unroll
        for (int m = 0; m < kMaps; ++m) d[m] = dots[m];
        const float4 pq = reinterpret_cast<const float4*>(o.Hpre)[t];
        const float4 oq = reinterpret_cast<const float4*>(o.Hpost)[t];
        const float hp[4] = {pq.x, pq.y, pq.z, pq.w};
        const float ho[4] = {oq.x, oq.y, oq.z, oq.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dl[j] = d[j] * hp[j] * (1.f - hp[j]);
            dl[4 + j] = d[4 + j] * ho[j] * (1.f - ho[j]);
        }
        float H[16];
        const float4* hr = reinterpret_cast<const float4*>(o.Hres + 16 * t);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 v = hr[q];
            H[4 * q] = v.x;
            H[4 * q + 1] = v.y;
            H[4 * q + 2] = v.z;
            H[4 * q + 3] = v.w;
        }
        project_bwd_refined(H, d + 8, dl + 8);
        // RMSNorm coefficient: <dl W, x / r> / (4C) = <dl, logits> / (4C)
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < kMaps; ++m) s = __builtin_fmaf(dl[m], o.logits[kMaps * t + m], s);
        o.svec[t] = s / (float)o.D;
        float4* go = reinterpret_cast<float4*>(o.glogits + kMaps * t);
#pragma unroll
        for (int q = 0; q < kMaps / 4; ++q) go[q] = make_float4(dl[4 * q], dl[4 * q + 1], dl[4 * q + 2], dl[4 * q + 3]);
        const float inv = 1.f / o.rms[t];
#pragma unroll
        for (int m = 0; m < kMaps; ++m) dl[m] *= inv;
    } else {
#pragma unroll
        for (int m = 0; m < kMaps; ++m) dl[m] = 0.f;
    }
#pragma unroll
    for (int m = 0; m < kMaps; ++m) {
        float v = dl[m];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const __bf16 h = (__bf16)v;
            o.dlT[dl_at(t, p, m)] = h;
            v -= (float)h;
        }
    }
}

template <int FMT, int W>
__global__ __launch_bounds__(kBlock) void layer_dots_ckpt_kernel(
    const uint2* __restrict__ xc, const uint8_t* __restrict__ xs, const uint2* __restrict__ fc,
    const uint8_t* __restrict__ fs, const uint4* __restrict__ gxo, const uint4* __restrict__ gu,
    DotsOut o, WtOut wt, int64_t Tp, int64_t C8, int tw)
{
    if (blockIdx.x >= wt.first) return transpose_W(wt, o.D);
    const int64_t T = o.T;
    __shared__ float sDots[4][16][kMaps];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t tb = ((int64_t)blockIdx.x * 4 + w) * tw;
    DotsLane L;
    L.xc = xc; L.xs = xs; L.fc = fc; L.fs = fs; L.gxo = gxo; L.gu = gu;
    L.T = T; L.C8 = C8; L.nch = (int)((C8 + W - 1) / W); L.tb = tb; L.lane = lane;
    float acc[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) acc[k] = 0.f;
    // the steps are taken in pairs; an odd last one is past the wave's tokens and does nothing
    DotsLoads d0, d1;
    DotsStep s0{0, 0};
    dots_issue<W>(L, d0, s0);
    const int n = tw / (64 / W);
    while (s0.tl < n) {
        const DotsStep s1 = dots_next(s0, L.nch), s2 = dots_next(s1, L.nch);
        dots_issue<W>(L, d1, s1);
        __builtin_amdgcn_sched_barrier(0);
        dots_consume<FMT, W>(L, d0, s0, acc, sDots[w]);
        __builtin_amdgcn_sched_barrier(0);
        dots_issue<W>(L, d0, s2);
        __builtin_amdgcn_sched_barrier(0);
        if (s1.tl < n) dots_consume<FMT, W>(L, d1, s1, acc, sDots[w]);
        __builtin_amdgcn_sched_barrier(0);
        s0 = s2;
    }
    __syncthreads();
    if (lane >= tw) return;
    const int64_t t = tb + lane;
    if (t >= Tp) return;
    finish_token(o, t, sDots[w][lane]);
}

// Few tokens of a wide layer: a workgroup per token, its 4 waves share the
// chunks (one wave per token walks 7168 columns in 14 dependent steps).
template <int FMT>
__global__ __launch_bounds__(kBlock) void layer_dots_few_ckpt_kernel(
    const uint2* __restrict__ xc, const uint8_t* __restrict__ xs, const uint2* __restrict__ fc,
    const uint8_t* __restrict__ fs, const uint4* __restrict__ gxo, const uint4* __restrict__ gu,
    DotsOut o, WtOut wt, int64_t C8)
{
    if (blockIdx.x >= wt.first) return transpose_W(wt, o.D);
    __shared__ float sDots[4][kMaps];
    __shared__ float sSum[kMaps];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t t = blockIdx.x;
    if (t < o.T) {
        DotsLane L;
        L.xc = xc; L.xs = xs; L.fc = fc; L.fs = fs; L.gxo = gxo; L.gu = gu;
        L.T = o.T; L.C8 = C8; L.tb = t; L.lane = lane;
        float acc[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[k] = 0.f;
        const int nch = (int)((C8 + 63) / 64);
        L.nch = nch + 1;  // no chunk is "the last": the reduction is here
        DotsLoads d0, d1;
        DotsStep s0{0, w};
        dots_issue<64>(L, d0, s0);
        while (s0.ci < nch) {
            const DotsStep s1{0, s0.ci + 4}, s2{0, s0.ci + 8};
            dots_issue<64>(L, d1, s1);
            __builtin_amdgcn_sched_barrier(0);
            dots_consume<FMT, 64>(L, d0, s0, acc, nullptr);
            __builtin_amdgcn_sched_barrier(0);
            dots_issue<64>(L, d0, s2);
            __builtin_amdgcn_sched_barrier(0);
            if (s1.ci < nch) dots_consume<FMT, 64>(L, d1, s1, acc, nullptr);
            __builtin_amdgcn_sched_barrier(0);
            s0 = s2;
        }
        const float sm = wave_sum_halving<32>(acc);
        const int idx = (lane >> 1) & 31;
        if ((lane & 1) == 0 && idx < kMaps) sDots[w][idx] = sm;
    }
    __syncthreads();
    if (threadIdx.x < kMaps)
        sSum[threadIdx.x] = (sDots[0][threadIdx.x] + sDots[1][threadIdx.x]) +
                            (sDots[2][threadIdx.x] + sDots[3][threadIdx.x]);
    __syncthreads();
    if (threadIdx.x == 0) finish_token(o, t, sSum);
}

// ---------------------------------------------------------------------------
// dx: workgroup = 16 tokens x a range of the columns (all of them unless the
// tokens are few), in chunks of 128 columns of every stream.  Bound by memory:
// 16384 x 7168 554-564 us, 5.0 TB/s.  Per chunk wave w forms (dl W)^T of stream
// w on MFMA (16 k x 16 tokens, A from the transposed W, B = dl in two bf16 parts, fixed for the
// workgroup) into LDS; then an element-wise pass with lane = (token, 8
// columns) whose accesses cover 4 rows x 256 contiguous bytes.  All loads of
// chunk i+1 are issued before chunk i is consumed, into the other of two
// register sets, and the LDS buffer is doubled, so one barrier per chunk
// suffices.
// ---------------------------------------------------------------------------
constexpr int kDxTok = 16;                    // tokens per workgroup (MFMA N)
constexpr int kDxChunk = 128;                 // columns per stream per chunk
constexpr int kDxTiles = kDxChunk / 16;       // k-tiles per wave per chunk
constexpr int kDxPitch = 4 * kDxChunk + 4;    // floats per LDS row (bank spread)

struct DxLoads {
    uint4 a[kDxTiles];    // transposed-W fragments of this wave's k-tiles
    uint4 g[4], u;        // grad_x_out, grad_u of the lane's token and columns
    uint2 x[4];           // checkpoint codes and scales of the same
    uint32_t sx[4];
};

struct DxLane {
    const uint2* xc;
    const uint8_t* xs;
    const uint4* gxo;
    const uint4* gu;
    const uint4* Wt;
    uint4* gx;
    uint4* gf;
    int64_t C, C8;
    int64_t tr;      // token row of the element-wise lane (clamped into range)
    bool tok;        // that token exists
    int w, row, kq, cl;
    float H[16], hp[4], ho[4], inv, sr;
    bf16x8 bhi, blo;
};

MHC_DEV void dx_issue(const DxLane& L, DxLoads& d, int64_t c0)
{
    // Wt rows past C (a ragged last chunk) are clamped; their products land
    // in LDS columns that the element-wise pass never reads.  Lanes kq = 3
    // (maps 24..31, which do not exist) load the piece of maps 0..7.
    const int kqc = L.kq < 3 ? L.kq : 0;
#pragma unroll
    for (int s = 0; s < kDxTiles; ++s) {
        int64_t c = c0 + 16 * s + L.row;
        c = c < L.C ? c : L.C - 1;
        d.a[s] = L.Wt[3 * (L.w * L.C + c) + kqc];
    }
    const bool col = c0 + 8 * L.cl < L.C;
    const int64_t c8 = col ? c0 / 8 + L.cl : L.C8 - 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        d.g[i] = L.gxo[(L.tr * 4 + i) * L.C8 + c8];
        d.x[i] = L.xc[(L.tr * 4 + i) * L.C8 + c8];
        d.sx[i] = L.xs[(L.tr * 4 + i) * (L.C8 / 4) + (c8 >> 2)];
    }
    d.u = L.gu[L.tr * L.C8 + c8];
}

template <int FMT>
MHC_DEV void dx_consume(const DxLane& L, const DxLoads& d, float (*sD)[kDxPitch], int64_t c0)
{
#pragma unroll
    for (int s = 0; s < kDxTiles; ++s) {
        // lanes kq = 3 hold a finite piece of another map range: their B
        // (maps 24..31) is zero, so they add nothing
        const bf16x8 a = as_bf16x8(d.a[s]);
        floatx4 acc = floatx4{0.f, 0.f, 0.f, 0.f};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, L.bhi, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, L.blo, acc, 0, 0, 0);
        *reinterpret_cast<floatx4*>(&sD[L.row][L.w * kDxChunk + 16 * s + 4 * L.kq]) = acc;
    }
    mhc_lds_barrier();
    const bool col = c0 + 8 * L.cl < L.C;
    if (!(L.tok && col)) return;
    const int tl = 4 * L.w + L.kq;  // element-wise token of this lane
    const int64_t c8 = c0 / 8 + L.cl;
    float gs[4][8], uu[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) mx_unpack8(d.g[i], gs[i]);
    mx_unpack8(d.u, uu);
    {
        float g8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float sm = L.ho[0] * gs[0][e];
            sm = __builtin_fmaf(L.ho[1], gs[1][e], sm);
            sm = __builtin_fmaf(L.ho[2], gs[2][e], sm);
            g8[e] = __builtin_fmaf(L.ho[3], gs[3][e], sm);
        }
        mhc_store_stream(&L.gf[L.tr * L.C8 + c8], mx_pack8(g8));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float xs[8], o8[8];
        mx_decode8<FMT>(d.x[j], mx_scale(d.sx[j]), xs);
        const floatx4 d0 = *reinterpret_cast<const floatx4*>(&sD[tl][j * kDxChunk + 8 * L.cl]);
        const floatx4 d1 = *reinterpret_cast<const floatx4*>(&sD[tl][j * kDxChunk + 8 * L.cl + 4]);
        const float dn[8] = {d0[0], d0[1], d0[2], d0[3], d1[0], d1[1], d1[2], d1[3]};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float sm = L.H[j] * gs[0][e];
            sm = __builtin_fmaf(L.H[4 + j], gs[1][e], sm);
            sm = __builtin_fmaf(L.H[8 + j], gs[2][e], sm);
            sm = __builtin_fmaf(L.H[12 + j], gs[3][e], sm);
            sm = __builtin_fmaf(L.hp[j], uu[e], sm);
            o8[e] = __builtin_fmaf(__builtin_fmaf(-xs[e], L.sr, dn[e]), L.inv, sm);
        }
        mhc_store_stream(&L.gx[(L.tr * 4 + j) * L.C8 + c8], mx_pack8(o8));
    }
}

template <int FMT>
__global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(2))) void layer_dx_ckpt_kernel(
    const uint2* __restrict__ xc, const uint8_t* __restrict__ xs, const uint4* __restrict__ gxo,
    const uint4* __restrict__ gu, const uint4* __restrict__ Wt, const float* __restrict__ Hpre,
    const float* __restrict__ Hpost, const float* __restrict__ Hres, const float* __restrict__ rms,
    const float* __restrict__ glogits, const float* __restrict__ svec, uint4* __restrict__ gx,
    uint4* __restrict__ gf, int64_t T, int64_t C, int64_t per)
{
    __shared__ __attribute__((aligned(16))) float sD[2][kDxTok][kDxPitch];
    DxLane L;
    const int lane = threadIdx.x & 63;
    L.xc = xc; L.xs = xs; L.gxo = gxo; L.gu = gu; L.Wt = Wt; L.gx = gx; L.gf = gf;
    L.C = C; L.C8 = C / 8;
    L.w = threadIdx.x >> 6;
    L.row = lane & 15;
    L.kq = lane >> 4;
    L.cl = lane & 15;
    const int64_t t0 = (int64_t)blockIdx.x * kDxTok;
    // B operand: dl[token t0 + row][maps 8 kq ..+7], two bf16 parts
    {
        float b8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) b8[e] = 0.f;
        if (t0 + L.row < T && L.kq < 3) {
            const float4* src = reinterpret_cast<const float4*>(glogits + kMaps * (t0 + L.row) + 8 * L.kq);
            const float4 v0 = src[0], v1 = src[1];
            b8[0] = v0.x; b8[1] = v0.y; b8[2] = v0.z; b8[3] = v0.w;
            b8[4] = v1.x; b8[5] = v1.y; b8[6] = v1.z; b8[7] = v1.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const __bf16 h = (__bf16)b8[e];
            L.bhi[e] = h;
            L.blo[e] = (__bf16)(b8[e] - (float)h);
        }
    }
    {
        const int64_t t = t0 + 4 * L.w + L.kq;
        L.tok = t < T;
        L.tr = L.tok ? t : T - 1;
        const float4* hr = reinterpret_cast<const float4*>(Hres + 16 * L.tr);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = hr[k];
            L.H[4 * k] = v.x;
            L.H[4 * k + 1] = v.y;
            L.H[4 * k + 2] = v.z;
            L.H[4 * k + 3] = v.w;
        }
        const float4 pq = reinterpret_cast<const float4*>(Hpre)[L.tr];
        L.hp[0] = pq.x; L.hp[1] = pq.y; L.hp[2] = pq.z; L.hp[3] = pq.w;
        const float4 oq = reinterpret_cast<const float4*>(Hpost)[L.tr];
        L.ho[0] = oq.x; L.ho[1] = oq.y; L.ho[2] = oq.z; L.ho[3] = oq.w;
        L.inv = 1.f / rms[L.tr];
        L.sr = svec[L.tr] * L.inv;
    }
    // branch-free pipeline: chunk counts are even, chunks past C load clamped
    // addresses and do no element-wise work
    const int64_t first = (int64_t)blockIdx.y * per;
    int64_t n = first + per;
    if (n * kDxChunk > C) n = (C + kDxChunk - 1) / kDxChunk;
    DxLoads d0, d1;
    dx_issue(L, d0, first * kDxChunk);
    for (int64_t ci = first; ci < n; ci += 2) {
        dx_issue(L, d1, (ci + 1) * kDxChunk);
        __builtin_amdgcn_sched_barrier(0);
        dx_consume<FMT>(L, d0, sD[0], ci * kDxChunk);
        __builtin_amdgcn_sched_barrier(0);
        dx_issue(L, d0, (ci + 2) * kDxChunk);
        __builtin_amdgcn_sched_barrier(0);
        dx_consume<FMT>(L, d1, sD[1], (ci + 1) * kDxChunk);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// ---------------------------------------------------------------------------
// dw: workgroup = 512 flattened k x one token group, a wave 128 of them:
//   dW^T tile (32 maps x 16 k) += dlT (32 maps x 32 tokens) * xhat (32 tokens x 16 k)
// Chunks of 32 tokens are copied straight from memory to LDS, two chunks ahead
// (with the loads in registers, one ahead, two waves per SIMD did not hide
// them: 16384 x 7168 162 us, so 112-120, the codes at 3.9-4.2 TB/s): a wave its own columns' codes and scales, all four the chunk's dlT,
// which lies together.  One barrier per chunk.
//
// The MFMA B operand wants 8 consecutive tokens of one k per lane, the memory
// holds 8 consecutive k of one token.  A lane reads 8 k of 8 tokens, decodes
// them to bf16 and transposes the 8 x 8 square in its own registers, two tokens
// at a time by byte permutes; MFMA tile nt then holds k = 8 (lane % 16) + nt
// instead of 16 consecutive k, which only relabels the columns of the result.
// One partial per token group is written, in a fixed order throughout.
// ---------------------------------------------------------------------------
constexpr int kDwK = 128;         // flattened k per wave
constexpr int kDwNt = kDwK / 16;  // MFMA tiles
constexpr int kDwStages = 3;
constexpr int kDlBytes = kDlParts * kMaps * 32 * 2;  // dlT of a chunk

struct DwStage {
    uint8_t x[4][32 * kDwK];  // a wave's codes: token r at row r ^ (r / 8 % 2), so that the rows
                              // a read covers (8 apart) fall on different banks
    uint32_t s[4][64];        // its scale bytes: 4 of a token in a word; half of it is used
    uint8_t dl[kDlBytes];
};

template <int FMT>
MHC_DEV void dw_consume(const DwStage& st, int w, int lane, floatx4 (&acc)[2][kDwNt])
{
    const int row = lane & 15, kq = lane >> 4;
    uint2 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = *reinterpret_cast<const uint2*>(&st.x[w][((8 * kq + e) ^ (kq & 1)) * kDwK + 8 * row]);
    uint32_t sc[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(&st.s[w][8 * kq + 4 * q]);
        sc[4 * q] = v.x;
        sc[4 * q + 1] = v.y;
        sc[4 * q + 2] = v.z;
        sc[4 * q + 3] = v.w;
    }
    bf16x8 a[kDlParts][2];  // maps 16 mt + row, tokens 8 kq ..+7
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
        const int m = 16 * mt + row < kMaps ? 16 * mt + row : kMaps - 1;
#pragma unroll
        for (int p = 0; p < kDlParts; ++p)
            a[p][mt] = as_bf16x8(*reinterpret_cast<const uint4*>(&st.dl[p * (kMaps * 64) + m * 64 + 16 * kq]));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 4 of the lane's 8 columns
        uint2 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = mx_decode4_bf16<FMT>(h ? x[e].y : x[e].x, mx_scale((sc[e] >> (8 * (row >> 2))) & 0xffu));
        bf16x8 bb[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t sel = q & 1 ? 0x07060302u : 0x05040100u;
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = q < 2 ? mx_perm(v[2 * i + 1].x, v[2 * i].x, sel) : mx_perm(v[2 * i + 1].y, v[2 * i].y, sel);
            bb[q] = as_bf16x8(make_uint4(b[0], b[1], b[2], b[3]));
        }
        // A rows 24..31 repeat map 23 (clamped load); they only feed D rows
        // 24..31, which are never stored.  Smallest parts first; the parts of
        // one tile are 8 products apart, so none waits for the one before.
#pragma unroll
        for (int p = kDlParts - 1; p >= 0; --p)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
                    acc[mt][4 * h + q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p][mt], bb[q], acc[mt][4 * h + q],
                                                                                0, 0, 0);
    }
}

template <int FMT>
__global__ __launch_bounds__(kBlock) void layer_dw_ckpt_kernel(
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs, const __bf16* __restrict__ dlT,
    float* __restrict__ partial, int64_t T, int64_t Tp, int64_t C, int64_t group_tokens)
{
    __shared__ __attribute__((aligned(16))) DwStage sS[kDwStages];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, kq = lane >> 4;
    const int64_t D = 4 * C;
    // waves past the width copy its last columns and store nothing
    const int64_t kw = (int64_t)blockIdx.x * (4 * kDwK) + kDwK * w, k0 = kw < D ? kw : D - kDwK;
    const int64_t g = blockIdx.y, tg0 = g * group_tokens;
    const int64_t tg1 = tg0 + group_tokens < Tp ? tg0 + group_tokens : Tp;
    const int chunks = (int)((tg1 - tg0) / 32);
    const uint32_t cD = (uint32_t)D, sD = cD / 32;
    const uint32_t lds = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)&sS[0]);
    constexpr int kCopies = 7;  // per wave and chunk
    // (chunks past the group's last one repeat it and are not used)
    const auto copy = [&](int ci, int buf) {
        const int64_t tc = tg0 + 32 * (int64_t)(ci < chunks ? ci : chunks - 1);
        // tokens past the last one repeat it: their dlT is zero
        const int64_t tb = tc < T ? tc : T - 1;
        const int last = (int)(T - tb < 32 ? T - tb : 32) - 1;
        const uint32_t at = lds + (uint32_t)sizeof(DwStage) * buf;
        const uint8_t* cb = xc + tb * D + k0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 8 tokens each
            int r = (8 * i + (lane >> 3)) ^ (i & 1);
            r = r < last ? r : last;
            copy16_to_lds(cb, (uint32_t)r * cD + 16u * (lane & 7), at + 32 * kDwK * w + 1024 * i);
        }
        int r = lane & 31;
        r = r < last ? r : last;
        copy4_to_lds(xs + (tb * D + k0) / 32, (uint32_t)r * sD, at + (uint32_t)offsetof(DwStage, s) + 256 * w);
        const uint8_t* db = reinterpret_cast<const uint8_t*>(dlT + dl_at(tc, 0, 0));
        const uint32_t dl = at + (uint32_t)offsetof(DwStage, dl);
        copy16_to_lds(db, 16u * (64 * w + lane), dl + 1024 * w);
        // the last 512 bytes; every wave, so that all count the same copies
        if (lane < 32) copy16_to_lds(db, 16u * (256 + lane), dl + 4096);
    };
    static_assert(kDlBytes == 4096 + 512, "dlT is copied by 4 waves and half a wave");
    floatx4 acc[2][kDwNt];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < kDwNt; ++nt) acc[mt][nt] = floatx4{0.f, 0.f, 0.f, 0.f};
    copy(0, 0);
    copy(1, 1);
    int buf = 0;
    for (int ci = 0; ci < chunks; ++ci) {
        // this chunk landed (the next one's copies may be under way), and
        // everybody has read the chunk before, whose buffer is next
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(kCopies) : "memory");
        copy(ci + 2, buf == 0 ? 2 : buf - 1);
        dw_consume<FMT>(sS[buf], w, lane, acc);
        buf = buf == 2 ? 0 : buf + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy outlives the workgroup
    if (kw >= D) return;
    float* out = partial + g * (int64_t)kMaps * D + k0 + 8 * row;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int m = 16 * mt + 4 * kq + v;
            if (m < kMaps) {
#pragma unroll
                for (int nt = 0; nt < kDwNt; nt += 4)
                    *reinterpret_cast<floatx4*>(&out[m * D + nt]) =
                        floatx4{acc[mt][nt][v], acc[mt][nt + 1][v], acc[mt][nt + 2][v], acc[mt][nt + 3][v]};
            }
        }
}

// grad_W from the partials: 4 threads to 4 columns, each a quarter of the
// groups, in a fixed order.
__global__ __launch_bounds__(kBlock) void layer_dw_sum_kernel(const float4* __restrict__ partial,
                                                              float4* __restrict__ gW, int64_t n4, int groups)
{
    __shared__ float4 sQ[4][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t i = (int64_t)blockIdx.x * 64 + lane;  // n4 is a multiple of 64
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int g = q; g < groups; g += 4) {
        const float4 v = partial[g * n4 + i];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    sQ[q][lane] = s;
    __syncthreads();
    if (q > 0) return;
    const float4 a = sQ[0][lane], b = sQ[1][lane], c = sQ[2][lane], d = sQ[3][lane];
    gW[i] = make_float4((a.x + b.x) + (c.x + d.x), (a.y + b.y) + (c.y + d.y), (a.z + b.z) + (c.z + d.z),
                        (a.w + b.w) + (c.w + d.w));
}

constexpr int64_t kFewTokens = 2048;

template <int FMT>
hipError_t layer_bwd_as(const LayerPtrs& a, const Packed& x, const Packed& f, int64_t T, int64_t C,
                        hipStream_t stream)
{
    const LayerCkptPlan p = layer_ckpt_plan(T, C);
    char* ws = static_cast<char*>(a.workspace);
    float* svec = reinterpret_cast<float*>(ws + p.off_s);
    __bf16* dlT = reinterpret_cast<__bf16*>(ws + p.off_dl);
    uint4* wt = reinterpret_cast<uint4*>(ws + p.off_wt);
    float* partial = reinterpret_cast<float*>(ws + p.off_partial);
    const uint2* xc = static_cast<const uint2*>(x.codes);
    const DotsOut o{a.H_pre, a.H_post, a.H_res, a.logits, a.rms, a.grad_logits, svec, dlT, T, 4 * C};
    const uint2* fc = static_cast<const uint2*>(f.codes);
    const uint4* gxo = static_cast<const uint4*>(a.grad_x_out);
    const uint4* gu = static_cast<const uint4*>(a.grad_u);
    const unsigned extra = (unsigned)((4 * C + kBlock - 1) / kBlock);
    WtOut wo{(const uint16_t*)a.W, wt, 0};
    if (T <= kFewTokens && C > 512) {
        wo.first = (unsigned)p.Tp;
        hipLaunchKernelGGL(layer_dots_few_ckpt_kernel<FMT>, dim3(wo.first + extra), dim3(kBlock), 0, stream,
                           xc, x.scales, fc, f.scales, gxo, gu, o, wo, C / 8);
    } else {
        int tw = 16;  // tokens per wave: a workgroup for every compute unit where there are as many tokens
        while (tw > (C <= 256 ? 4 : 1) && p.Tp / (4 * tw) < 256) tw /= 2;
        wo.first = (unsigned)(p.Tp / (4 * tw));
        auto* dots = C <= 256 ? layer_dots_ckpt_kernel<FMT, 16> : layer_dots_ckpt_kernel<FMT, 64>;
        hipLaunchKernelGGL(dots, dim3(wo.first + extra), dim3(kBlock), 0, stream, xc, x.scales, fc, f.scales,
                           gxo, gu, o, wo, p.Tp, C / 8, tw);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // column ranges of whole pairs of chunks, for about 512 workgroups
    const int64_t tiles = (T + kDxTok - 1) / kDxTok, pairs = (C + 2 * kDxChunk - 1) / (2 * kDxChunk);
    int64_t ranges = (512 + tiles - 1) / tiles;
    ranges = ranges < pairs ? ranges : pairs;
    const int64_t per = 2 * ((pairs + ranges - 1) / ranges);
    ranges = (2 * pairs + per - 1) / per;
    hipLaunchKernelGGL(layer_dx_ckpt_kernel<FMT>, dim3((unsigned)tiles, (unsigned)ranges), dim3(kBlock), 0,
                       stream, xc, x.scales, gxo, gu, wt, a.H_pre, a.H_post, a.H_res, a.rms,
                       a.grad_logits, svec, (uint4*)a.grad_x, (uint4*)a.grad_f, T, C, per);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(layer_dw_ckpt_kernel<FMT>, dim3((unsigned)((4 * C + 4 * kDwK - 1) / (4 * kDwK)), (unsigned)p.groups),
                       dim3(kBlock), 0, stream, (const uint8_t*)x.codes, x.scales, dlT,
                       p.groups == 1 ? a.grad_W : partial, T, p.Tp, C, p.group_tokens);
    e = hipGetLastError();
    if (e != hipSuccess || p.groups == 1) return e;
    const int64_t n4 = kMaps * C;  // of 4 columns
    hipLaunchKernelGGL(layer_dw_sum_kernel, dim3((unsigned)(n4 / 64)), dim3(kBlock), 0, stream,
                       (const float4*)partial, (float4*)a.grad_W, n4, (int)p.groups);
    return hipGetLastError();
}

template <int FMT>
hipError_t layer_finish_as(const LayerPtrs& a, const Packed& x, const Packed& f, const ReadPlan& p, int64_t T,
                           int64_t C, float eps, const SolverOpts& o, hipStream_t stream)
{
    const TokenMaps maps{a.logits, a.rms, a.H_pre, a.H_post, a.H_res};
    auto* kernel = o.solver == 0 ? layer_finish_ckpt_kernel<0, FMT> : layer_finish_ckpt_kernel<1, FMT>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)T), dim3(kBlock), 0, stream, (const uint4*)a.x, (const uint4*)a.f,
                       static_cast<const float*>(a.workspace), (int)p.splits, maps, (uint4*)a.u, (uint4*)a.x_out,
                       (uint2*)x.codes, x.scales, (uint2*)f.codes, f.scales, T, C / 8, eps, o);
    return hipGetLastError();
}

template <int FMT>
hipError_t layer_mix_as(const LayerPtrs& a, const Packed& x, const Packed& f, int64_t T, int64_t C,
                        hipStream_t stream)
{
    const int shift = token_shift(C / 8);
    auto* kernel = shift < 6 ? layer_mix_ckpt_kernel<FMT, true> : layer_mix_ckpt_kernel<FMT, false>;
    hipLaunchKernelGGL(kernel, dim3(token_grid(T)), dim3(kBlock), 0, stream, (const uint4*)a.x,
                       (const uint4*)a.f, a.H_pre, a.H_post, a.H_res, (uint4*)a.u, (uint4*)a.x_out,
                       (uint2*)x.codes, x.scales, (uint2*)f.codes, f.scales, T, C / 8, shift);
    return hipGetLastError();
}

}  // namespace

LayerCkptPlan layer_ckpt_plan(int64_t T, int64_t C)
{
    LayerCkptPlan p;
    p.Tp = layer_plan(T, C).Tp;
    // token groups of the grad_W pass: one round of workgroups, two to a
    // compute unit, but 64 groups at most (their partials are read back)
    const int64_t columns = (4 * C + 4 * kDwK - 1) / (4 * kDwK);
    int64_t want = 512 / columns;
    want = want < 1 ? 1 : (want > 64 ? 64 : want);
    if (p.Tp <= 256) want = 1;  // straight to grad_W
    p.group_tokens = ((p.Tp + want - 1) / want + 63) / 64 * 64;
    if (p.group_tokens < 64) p.group_tokens = 64;  // no tokens
    p.groups = (p.Tp + p.group_tokens - 1) / p.group_tokens;
    const int64_t D = 4 * C;
    p.off_s = 0;
    p.off_dl = (p.Tp * 4 + 255) / 256 * 256;
    p.off_wt = p.off_dl + (p.Tp * kMaps * 2 * kDlParts + 255) / 256 * 256;
    p.off_partial = p.off_wt + (D * kMaps * 2 + 255) / 256 * 256;
    p.bytes = p.off_partial + p.groups * kMaps * D * 4;
    return p;
}

hipError_t launch_layer_fwd_ckpt(const LayerPtrs& a, const Packed& x, const Packed& f, int64_t T,
                                 int64_t C, float eps, int fmt, const SolverOpts& o,
                                 hipStream_t stream)
{
    const ReadPlan p = read_plan(T, C);
    if (p.splits != 0) {
        const hipError_t e = launch_read_part(a, p, T, C, stream);
        if (e != hipSuccess) return e;
        return fmt == kE4M3 ? layer_finish_as<kE4M3>(a, x, f, p, T, C, eps, o, stream)
                            : layer_finish_as<kInt8>(a, x, f, p, T, C, eps, o, stream);
    }
    const hipError_t e = launch_layer_maps(a, T, C, eps, o, stream);
    if (e != hipSuccess) return e;
    return fmt == kE4M3 ? layer_mix_as<kE4M3>(a, x, f, T, C, stream)
                        : layer_mix_as<kInt8>(a, x, f, T, C, stream);
}

hipError_t launch_layer_bwd_ckpt(const LayerPtrs& a, const Packed& x, const Packed& f, int64_t T,
                                 int64_t C, int fmt, hipStream_t stream)
{
    return fmt == kE4M3 ? layer_bwd_as<kE4M3>(a, x, f, T, C, stream)
                        : layer_bwd_as<kInt8>(a, x, f, T, C, stream);
}

}  // namespace mhc
