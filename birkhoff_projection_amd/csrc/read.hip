// The read half of the residual-layer step (layer.hip) on its own, for gfx950:
// the token's maps and the layer function's input u = sum_j H_pre[j] x_j, as
// bf16 or quantised to MXFP4 (mxfmt.h) in the same pass.
//
// Many tokens: the layer's maps pass, then one pass over x for u (16384 x 4096:
// 128-133 us, 4.0-4.2 TB/s, and 84 us; x is read twice, the second time in part
// from the cache).
//
// Few tokens: that maps pass runs one workgroup per 64 tokens, each walking
// the whole width 4C, so a single token would take as long as 16384.  Here
// the width is split over the grid instead:
//   part    16 tokens x one piece of the width per workgroup: MFMA partial
//           logits and sums of squares, written as partials [S][T][25]
//   finish  one workgroup per token: the partials summed in a fixed order,
//           maps and projection, then u (the projection runs in one wave
//           while the others go on to u, which does not need it)
// One token of 4096: 4.6 and 6.5 us, two dependent kernels; an empty one takes
// 2-2.5.
#include "mxfmt.h"
#include "proj4.h"
#include "qkernels.h"
#include "tokenmaps.h"
#include "wave.h"

namespace mhc {

namespace {

constexpr int kBlock = 256;
constexpr int kMaps = kTokenMaps, kVals = kTokenVals;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

// u of 8 columns, stored as bf16 and / or MXFP4.  The 4-bit codes are those of
// the bf16 u, so they do not depend on whether u itself is kept.  Quads of
// lanes must be whole.
struct UOut {
    uint4* u;          // [T, C] bf16 or NULL
    uint32_t* codes;   // [T, C/2] or NULL
    uint8_t* scales;   // [T, C/32]
};

MHC_DEV void store_u(const UOut& o, int64_t i, const float (&M)[4], const uint4 (&xq)[4])
{
    float xs[4][8], uu[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) mx_unpack8(xq[j], xs[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float s = M[0] * xs[0][e];
        s = __builtin_fmaf(M[1], xs[1][e], s);
        s = __builtin_fmaf(M[2], xs[2][e], s);
        uu[e] = __builtin_fmaf(M[3], xs[3][e], s);
    }
    const uint4 q = mx_pack8(uu);
    if (o.u != nullptr) mhc_store_stream(&o.u[i], q);
    if (o.codes != nullptr) {
        const uint32_t amax = mx_quad_max(mx_amax8(q)), s = mx_scale_byte<kE2M1>(amax);
        o.codes[i] = mx_encode8_e2m1(q, amax, s);
        if ((i & 3) == 0) o.scales[i >> 2] = (uint8_t)s;
    }
}

// u for many tokens: 16 tokens per workgroup, spaced by the grid size.
constexpr int kMixTokens = 16;

template <bool NARROW>
__global__ __launch_bounds__(kBlock) void read_mix_kernel(const uint4* __restrict__ x,
                                                          const float* __restrict__ Hpre, UOut o,
                                                          int64_t T, int64_t C8, int shift)
{
    const int64_t b = blockIdx.x, G = gridDim.x;
    const int tid = threadIdx.x;
    // 2^shift threads share a token
    for (int tl = first_token<NARROW>(tid, shift); tl < kMixTokens; tl += kBlock >> shift) {
        const int64_t t = b + G * tl;
        if (t >= T) return;
        const float4 h = reinterpret_cast<const float4*>(Hpre)[t];
        const float M[4] = {h.x, h.y, h.z, h.w};
        // C8 is a multiple of 8: a quad of lanes (one block) is whole
        for (int64_t c = tid & ((1 << shift) - 1); c < C8; c += 1 << shift) {
            uint4 xq[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) xq[j] = mhc_load_stream(&x[(t * 4 + j) * C8 + c]);
            store_u(o, t * C8 + c, M, xq);
        }
    }
}

// Partial logits of NT tiles of 16 tokens: 4 waves take the 32-wide steps of
// the workgroup's piece of the width in turn.  MFMA 16x16x32: A = x rows (token
// l % 16, k 8 (l / 16)), B = W rows (map l % 16), D lane l, v: token
// 4 (l / 16) + v, map l % 16.  Each step of W comes from the caches anew, half
// again as many bytes as x of one tile: with enough tokens NT is 4.
constexpr int kPartTok = 16;

template <int NT>
__global__ __launch_bounds__(kBlock) void read_part_kernel(const uint16_t* __restrict__ x,
                                                           const uint16_t* __restrict__ W,
                                                           float* __restrict__ partial, int64_t T,
                                                           int64_t D, int64_t steps_per)
{
    constexpr int kTok = kPartTok * NT;
    __shared__ float sR[4][kTok][kMaps + 1];
    __shared__ float sQ[4][kTok];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int row = lane & 15, kq = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * kTok;
    const uint16_t* xp[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t t = t0 + kPartTok * j + row;
        xp[j] = x + (t < T ? t : T - 1) * D + 8 * kq;
    }
    const uint16_t* w0 = W + row * D + 8 * kq;
    const uint16_t* w1 = W + (16 + (row & 7)) * D + 8 * kq;  // maps 16..23, twice
    const int64_t s0 = (int64_t)blockIdx.y * steps_per;
    int64_t s1 = s0 + steps_per;
    s1 = s1 < D / 32 ? s1 : D / 32;
    floatx4 acc0[NT], acc1[NT];
    float ssq[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        acc0[j] = floatx4{0.f, 0.f, 0.f, 0.f};
        acc1[j] = acc0[j];
        ssq[j] = 0.f;
    }
    constexpr int kAhead = 4;  // steps' loads at once
    for (int64_t s = s0 + w; s < s1; s += 4 * kAhead) {
        uint4 a[kAhead][NT], b0[kAhead], b1[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t at = s + 4 * i < s1 ? s + 4 * i : s;
#pragma unroll
            for (int j = 0; j < NT; ++j) a[i][j] = *reinterpret_cast<const uint4*>(xp[j] + 32 * at);
            b0[i] = *reinterpret_cast<const uint4*>(w0 + 32 * at);
            b1[i] = *reinterpret_cast<const uint4*>(w1 + 32 * at);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s + 4 * i >= s1) break;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc0[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, a[i][j]), __builtin_bit_cast(bf16x8, b0[i]), acc0[j], 0, 0, 0);
                acc1[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, a[i][j]), __builtin_bit_cast(bf16x8, b1[i]), acc1[j], 0, 0, 0);
                float f[8];
                mx_unpack8(a[i][j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) ssq[j] = __builtin_fmaf(f[e], f[e], ssq[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            float* d = sR[w][kPartTok * j + 4 * kq + v];
            d[row] = acc0[j][v];
            if (row < 8) d[16 + row] = acc1[j][v];
        }
        const float q = sum_bit5(sum_bit4(ssq[j]));
        if (kq == 0) sQ[w][kPartTok * j + row] = q;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < kTok * kVals; p += kBlock) {
        const int tl = p / kVals, m = p % kVals;
        if (t0 + tl >= T) break;
        const float v = m < kMaps ? (sR[0][tl][m] + sR[1][tl][m]) + (sR[2][tl][m] + sR[3][tl][m])
                                  : (sQ[0][tl] + sQ[1][tl]) + (sQ[2][tl] + sQ[3][tl]);
        partial[((int64_t)blockIdx.y * T + t0 + tl) * kVals + m] = v;
    }
}

template <int SOLVER>
__global__ __launch_bounds__(kBlock) void read_finish_kernel(
    const uint4* __restrict__ x, const float* __restrict__ partial, int splits, TokenMaps maps, UOut o,
    int64_t T, int64_t C8, float eps, SolverOpts opts)
{
    __shared__ TokenLds s;
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    const float inv = token_logits(s, partial, splits, maps, t, T, C8, eps);
    if (tid < 64) {  // wave 0: the projection (one lane), the others go on to u
        float h[16];
        if (tid == 0) token_project<SOLVER>(s, inv, maps, t, opts, h);
        return;
    }
    float M[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) M[j] = token_sigmoid(s.l[j] * inv);
    for (int64_t c = tid - 64; c < C8; c += kBlock - 64) {
        uint4 xq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) xq[j] = x[(t * 4 + j) * C8 + c];
        store_u(o, t * C8 + c, M, xq);
    }
}

}  // namespace

// Up to kReadFewTokens tokens take the split kernels, and up to
// kReadFewWideTokens of rows wide enough: about 512 workgroups in all (1024
// are no faster) of at least 16 steps of 32 (4 per wave) each.  Maps and u, us,
// against the maps pass over whole rows, whose workgroups then are few: 4096 x
// 7168 87 / 155, 8192 x 7168 201 / 210, 8192 x 2048 58 / 65; but 8192 x 1024
// 43 / 36 and 4096 x 512 24 / 18 (a workgroup per token for the second half).
constexpr int64_t kReadFewTokens = 2048, kReadFewWideTokens = 8192, kReadWide = 2048;

ReadPlan read_plan(int64_t T, int64_t C)
{
    ReadPlan p{0, 0, 0, 1};
    if (T <= 0 || T > (C >= kReadWide ? kReadFewWideTokens : kReadFewTokens)) return p;
    p.tiles = T >= 512 ? 4 : 1;
    const int64_t steps = 4 * C / 32, groups = (T + kPartTok * p.tiles - 1) / (kPartTok * p.tiles);
    int64_t want = (512 + groups - 1) / groups;
    if (want > steps / 16) want = steps / 16;
    if (want < 1) want = 1;
    p.steps_per = (steps + want - 1) / want;
    p.splits = (steps + p.steps_per - 1) / p.steps_per;
    p.bytes = p.splits * T * kVals * 4;
    return p;
}

hipError_t launch_read_part(const LayerPtrs& a, const ReadPlan& p, int64_t T, int64_t C, hipStream_t stream)
{
    const int64_t tok = kPartTok * p.tiles;
    auto* part = p.tiles == 4 ? read_part_kernel<4> : read_part_kernel<1>;
    hipLaunchKernelGGL(part, dim3((unsigned)((T + tok - 1) / tok), (unsigned)p.splits), dim3(kBlock), 0,
                       stream, (const uint16_t*)a.x, (const uint16_t*)a.W, static_cast<float*>(a.workspace), T,
                       4 * C, p.steps_per);
    return hipGetLastError();
}

hipError_t launch_layer_read(const LayerPtrs& a, const Packed& u4, int64_t T, int64_t C, float eps,
                             const SolverOpts& o, hipStream_t stream)
{
    const UOut uo{(uint4*)a.u, (uint32_t*)u4.codes, u4.scales};
    const ReadPlan p = read_plan(T, C);
    if (p.splits != 0) {
        const hipError_t e = launch_read_part(a, p, T, C, stream);
        if (e != hipSuccess) return e;
        const TokenMaps maps{a.logits, a.rms, a.H_pre, a.H_post, a.H_res};
        auto* finish = o.solver == 0 ? read_finish_kernel<0> : read_finish_kernel<1>;
        hipLaunchKernelGGL(finish, dim3((unsigned)T), dim3(kBlock), 0, stream, (const uint4*)a.x,
                           static_cast<const float*>(a.workspace), (int)p.splits, maps, uo, T, C / 8, eps, o);
        return hipGetLastError();
    }
    const hipError_t e = launch_layer_maps(a, T, C, eps, o, stream);
    if (e != hipSuccess) return e;
    const int shift = token_shift(C / 8);
    auto* kernel = shift < 6 ? read_mix_kernel<true> : read_mix_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(token_grid(T)), dim3(kBlock), 0, stream, (const uint4*)a.x,
                       a.H_pre, uo, T, C / 8, shift);
    return hipGetLastError();
}

}  // namespace mhc
