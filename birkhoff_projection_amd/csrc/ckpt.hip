// Packing activations into blocks of 32 with a shared scale (mxfmt.h), and
// the stream mix that keeps its input as such a checkpoint, for gfx950.
//
//   pack / unpack      bf16 or fp32 rows <-> 8-bit (or 4-bit) codes + scales
//   transposed pack    4-bit codes along the columns of a row-major matrix:
//                      the operand of a product that sums over its rows
//   mix forward        out_i = sum_j H_ij x_j, and x packed in the same pass
//   mix backward       grad_x_j = sum_i H_ij g_i, grad_H_ij = <g_i, xhat_j>
//                      with xhat the packed x
//
// All of them move each byte once; a lane moves 8 columns (16 bytes of bf16, 8
// or 4 bytes of codes), consecutive lanes take consecutive columns.  Along the
// rows they are bound by HBM: pack and unpack 65536 x 7168 221 and 228 us
// (6.3 TB/s), 4-bit rows of 16384 x 7168 46 us, of 8192 x 4096 15 (5.7 TB/s);
// mix 16384 x 4096 forward 240 us, backward 246 (5.5 TB/s).  Along the columns
// 16384 x 7168 takes 53-60 us (5 TB/s), both 90, columns from a checkpoint 42
// (4.4), but few tiles do not reach that rate: columns of 8192 x 4096 26 us
// (3.2 TB/s), both of 8192 x 8192 57 (3.6), from a checkpoint 8192 x 4096 18
// (2.9).  A tile's workgroup loads all, then stores all, and there is little
// more than one round of workgroups to overlap the two.
#include "mxfmt.h"
#include "proj4.h"
#include "qkernels.h"
#include "wave.h"

namespace mhc {

namespace {

constexpr int kBlock = 256;
constexpr int kUnroll = 4;                       // chunks of 8 columns per lane
constexpr int kWaveChunks = 64 * kUnroll;

// Chunk p of the packed order (rows padded to whole blocks) -> chunk of the
// unpadded rows; false past a row's end.  RAG: the width is no multiple of 32.
template <bool RAG>
MHC_DEV bool chunk_of(int64_t row0, uint32_t q, uint32_t P8, uint32_t C8, int64_t p, int64_t* off)
{
    if (!RAG) {
        *off = p;
        return true;
    }
    const uint32_t r = q / P8, c = q - r * P8;
    const bool in = c < C8;
    *off = (row0 + r) * C8 + (in ? c : C8 - 1);
    return in;
}

// ---------------------------------------------------------------------------
// pack: a wave takes 256 chunks in 4 loads per lane, all issued first.  The
// 64 scale bytes of a wave are gathered in LDS and leave as one 64-byte
// store.  AND4: an 8-bit pack that writes the 4-bit one as well.
// ---------------------------------------------------------------------------
template <int FMT, bool F32, bool RAG, bool AND4 = false>
__global__ __launch_bounds__(kBlock) void pack_kernel(const uint4* __restrict__ x,
                                                      void* __restrict__ codes,
                                                      uint8_t* __restrict__ scales,
                                                      uint32_t* __restrict__ codes4,
                                                      uint8_t* __restrict__ scales4, int64_t n,
                                                      uint32_t P8, uint32_t C8)
{
    __shared__ __attribute__((aligned(16))) uint8_t sS[kBlock / 64][kWaveChunks / 4];
    __shared__ __attribute__((aligned(16))) uint8_t sS4[AND4 ? kBlock / 64 : 1][kWaveChunks / 4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t base = ((int64_t)blockIdx.x * (kBlock / 64) + w) * kWaveChunks;
    if (base >= n) return;
    int64_t row0 = 0;
    uint32_t rem0 = 0;
    if (RAG) {
        row0 = base / P8;
        rem0 = (uint32_t)(base - row0 * P8);
    }
    uint4 v[kUnroll][F32 ? 2 : 1];
    int64_t off[kUnroll];
    bool in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        // chunks past the end repeat the last one and are not stored; the
        // packed order ends with a whole block, so a quad of lanes is whole
        int64_t p = base + 64 * u + lane;
        const bool live = p < n;
        p = live ? p : n - 1;
        in[u] = chunk_of<RAG>(row0, rem0 + (uint32_t)(p - base), P8, C8, p, &off[u]) && live;
#pragma unroll
        for (int h = 0; h < (F32 ? 2 : 1); ++h) v[u][h] = mhc_load_stream(&x[(F32 ? 2 : 1) * off[u] + h]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (RAG && !in[u]) {
#pragma unroll
            for (int h = 0; h < (F32 ? 2 : 1); ++h) v[u][h] = make_uint4(0, 0, 0, 0);
        }
        float f[8];
        uint32_t amax;
        if (F32) {
            const float4 a = __builtin_bit_cast(float4, v[u][0]);
            const float4 b = __builtin_bit_cast(float4, v[u][F32 ? 1 : 0]);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            amax = mx_amax8(f);
        } else {
            amax = mx_amax8(v[u][0]);
        }
        amax = mx_quad_max(amax);
        const uint32_t s = mx_scale_byte<FMT>(amax);
        if constexpr (AND4) {
            const uint32_t s4 = mx_scale_byte<kE2M1>(amax);
            float f4[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f4[e] = F32 ? f[e] : 0.f;
            const uint32_t c4 = F32 ? mx_encode8_e2m1(f4, amax, s4) : mx_encode8_e2m1(v[u][0], amax, s4);
            if (in[u]) codes4[off[u]] = c4;
            if ((lane & 3) == 0) sS4[w][16 * u + (lane >> 2)] = (uint8_t)s4;
        }
        if (FMT == kE2M1) {
            const uint32_t c = F32 ? mx_encode8_e2m1(f, amax, s) : mx_encode8_e2m1(v[u][0], amax, s);
            if (in[u]) reinterpret_cast<uint32_t*>(codes)[off[u]] = c;
        } else {
            if (!F32) mx_unpack8(v[u][0], f);
            const uint2 c = mx_encode8<FMT>(f, amax, s);
            if (in[u]) mx_store_stream(reinterpret_cast<uint2*>(codes) + off[u], c);
        }
        if ((lane & 3) == 0) sS[w][16 * u + (lane >> 2)] = (uint8_t)s;
    }
    mhc_wave_lds_fence();
    const auto store_scales = [&](uint8_t* all, const uint8_t* from) {
        uint8_t* dst = all + base / 4;
        if (base + kWaveChunks <= n) {
            if (lane < 16) reinterpret_cast<uint32_t*>(dst)[lane] = *reinterpret_cast<const uint32_t*>(&from[4 * lane]);
        } else if (base + 4 * lane < n) {
            dst[lane] = from[lane];
        }
    };
    store_scales(scales, sS[w]);
    if constexpr (AND4) store_scales(scales4, sS4[w]);
}

template <int FMT, bool F32, bool RAG>
__global__ __launch_bounds__(kBlock) void unpack_kernel(const void* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales,
                                                        uint4* __restrict__ x, int64_t n,
                                                        uint32_t P8, uint32_t C8)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t base = ((int64_t)blockIdx.x * (kBlock / 64) + w) * kWaveChunks;
    if (base >= n) return;
    int64_t row0 = 0;
    uint32_t rem0 = 0;
    if (RAG) {
        row0 = base / P8;
        rem0 = (uint32_t)(base - row0 * P8);
    }
    uint2 c[kUnroll];
    uint32_t s[kUnroll];
    int64_t off[kUnroll];
    bool in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        int64_t p = base + 64 * u + lane;
        const bool live = p < n;
        p = live ? p : n - 1;
        in[u] = chunk_of<RAG>(row0, rem0 + (uint32_t)(p - base), P8, C8, p, &off[u]) && live;
        if (FMT == kE2M1)
            c[u] = make_uint2(reinterpret_cast<const uint32_t*>(codes)[off[u]], 0u);
        else
            c[u] = mx_load_stream(reinterpret_cast<const uint2*>(codes) + off[u]);
        s[u] = scales[p / 4];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        float f[8];
        if (FMT == kE2M1)
            mx_decode8_e2m1(c[u].x, mx_scale(s[u]), f);
        else
            mx_decode8<FMT>(c[u], mx_scale(s[u]), f);
        if (!in[u]) continue;
        if (F32) {
            mhc_store_stream(&x[2 * off[u]], __builtin_bit_cast(uint4, make_float4(f[0], f[1], f[2], f[3])));
            mhc_store_stream(&x[2 * off[u] + 1], __builtin_bit_cast(uint4, make_float4(f[4], f[5], f[6], f[7])));
        } else {
            mhc_store_stream(&x[off[u]], mx_pack8(f));
        }
    }
}

// ---------------------------------------------------------------------------
// Transposed 4-bit pack: x [R, C] -> codes [C, R/2], scales [C, R/32], blocks
// of 32 rows of one column.  A workgroup takes 256 rows x 64 columns; a lane
// takes 2 adjacent columns of 32 rows, so its two block maxima and all codes
// stay in the lane, and each load instruction covers 64 columns of 2 rows.
// The codes go through LDS so that a column's 128 bytes leave together.
// ROWS: the rows are packed as well, from a copy of the tile in LDS; a lane
// then takes 8 columns of a row, as in pack.  One read of x instead of two.
// Tiles of one band of rows run one after the other on one die, so that the
// 32 bytes of codes of each tile's row meet in its cache.
// ---------------------------------------------------------------------------
constexpr int kTrRows = 256, kTrCols = 64;
constexpr int kTrPitch = kTrRows / 2 + 16;  // bytes per column of codes in LDS

// 32 rows of two adjacent columns (bf16 pairs) to codes and scale bytes, the
// second column's `pitch` and `spitch` bytes behind the first's.
MHC_DEV void pack_column_pair(const uint32_t (&v)[32], uint8_t* codes, int pitch, uint8_t* scale, int spitch)
{
    mx_u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 32; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_u16x2, v[i] & 0x7fff7fffu));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t amax = (uint32_t)(k ? m.y : m.x) << 16, sel = k ? 0x07060302u : 0x05040100u;
        const uint32_t s = mx_scale_byte<kE2M1>(amax);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = mx_encode8_e2m1(make_uint4(mx_perm(v[8 * i + 1], v[8 * i], sel),
                                              mx_perm(v[8 * i + 3], v[8 * i + 2], sel),
                                              mx_perm(v[8 * i + 5], v[8 * i + 4], sel),
                                              mx_perm(v[8 * i + 7], v[8 * i + 6], sel)), amax, s);
        *reinterpret_cast<uint4*>(codes + k * pitch) = make_uint4(o[0], o[1], o[2], o[3]);
        scale[k * spitch] = (uint8_t)s;
    }
}

// A tile's columns of codes and scales from LDS to memory.
template <int COLS>
MHC_DEV void store_columns(const uint8_t (*sC)[kTrPitch], const uint8_t (*sS)[kTrRows / 32],
                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t r0,
                           int64_t c0, int64_t R, int64_t C)
{
    const int tid = threadIdx.x;
    const int nb = (int)(R - r0 < kTrRows ? (R - r0) / 32 : kTrRows / 32);  // row blocks here
#pragma unroll
    for (int i = 0; i < COLS * 8 / kBlock; ++i) {
        const int p = tid + kBlock * i, col = p >> 3, b = p & 7;
        if (c0 + col < C && b < nb)
            *reinterpret_cast<uint4*>(codes + (c0 + col) * (R / 2) + r0 / 2 + 16 * b) =
                *reinterpret_cast<const uint4*>(&sC[col][16 * b]);
    }
#pragma unroll
    for (int i = 0; i < COLS * 8 / kBlock; ++i) {
        const int p = tid + kBlock * i, col = p >> 3, b = p & 7;
        if (c0 + col < C && b < nb) scales[(c0 + col) * (R / 32) + r0 / 32 + b] = sS[col][b];
    }
}

template <bool F32, bool ROWS>
__global__ __launch_bounds__(kBlock) void pack_transposed_kernel(
    const void* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
    uint32_t* __restrict__ row_codes, uint8_t* __restrict__ row_scales, int64_t R, int64_t C)
{
    constexpr int kRowWords = kTrCols * (F32 ? 4 : 2) / 4;  // of the copy
    __shared__ __attribute__((aligned(16))) uint8_t sC[kTrCols][kTrPitch];
    __shared__ __attribute__((aligned(8))) uint8_t sS[kTrCols][kTrRows / 32];
    __shared__ __attribute__((aligned(16))) uint32_t sV[ROWS ? kTrRows : 1][kRowWords];
    const int tid = threadIdx.x;
    const int cp = tid & 31, rb = tid >> 5;   // column pair, row block of 32
    int64_t bx = blockIdx.x, by = blockIdx.y;
    if (ROWS) {  // a linear grid: column tiles fastest, each die a run of tiles
        const unsigned total = gridDim.x, per = total / 8, extra = total % 8, die = blockIdx.x % 8;
        const unsigned t = die * per + (die < extra ? die : extra) + blockIdx.x / 8;
        const unsigned gc = (unsigned)((C + kTrCols - 1) / kTrCols);
        bx = t / gc;
        by = t % gc;
    }
    const int64_t r0 = bx * kTrRows, c0 = by * kTrCols;
    const int64_t r = r0 + 32 * rb;
    int64_t c = c0 + 2 * cp;
    c = c < C ? c : C - 2;                    // columns past the end: loaded, not stored
    // row i of the tile is at row i ^ (i / 32 % 2) of the copy: a wave writes
    // rows i and i + 32 at once, which so fall on different banks
    if (r < R) {                              // R is a multiple of 32: a block is whole
        if constexpr (F32) {
            const float* p = reinterpret_cast<const float*>(x) + r * C + c;
            float f[2][32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float2 v = *reinterpret_cast<const float2*>(p + i * C);
                f[0][i] = v.x;
                f[1][i] = v.y;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t amax = 0;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    const uint32_t m = mx_amax8(&f[k][i]);
                    amax = m > amax ? m : amax;
                }
                if constexpr (ROWS)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sV[32 * rb + (i ^ (rb & 1))][2 * cp + k] = __float_as_uint(f[k][i]);
                const uint32_t s = mx_scale_byte<kE2M1>(amax);
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = mx_encode8_e2m1(&f[k][8 * i], amax, s);
                *reinterpret_cast<uint4*>(&sC[2 * cp + k][16 * rb]) = make_uint4(o[0], o[1], o[2], o[3]);
                sS[2 * cp + k][rb] = (uint8_t)s;
            }
        } else {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(x) + r * C + c;
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = *reinterpret_cast<const uint32_t*>(p + i * C);
            if constexpr (ROWS)
#pragma unroll
                for (int i = 0; i < 32; ++i) sV[32 * rb + (i ^ (rb & 1))][cp] = v[i];
            pack_column_pair(v, &sC[2 * cp][16 * rb], kTrPitch, &sS[2 * cp][rb], kTrRows / 32);
        }
    }
    __syncthreads();
    store_columns<kTrCols>(sC, sS, codes, scales, r0, c0, R, C);
    if constexpr (ROWS) {
        // 16 columns per lane, a block per pair of lanes; C is a multiple of 32
#pragma unroll
        for (int j = 0; j < kTrRows * 4 / kBlock; ++j) {
            const int p = tid + kBlock * j, row = p >> 2, c16 = p & 3;
            const int64_t rr = r0 + row, cc = c0 + 16 * c16;
            const uint4* q = reinterpret_cast<const uint4*>(&sV[row ^ ((row >> 5) & 1)][kRowWords / 4 * c16]);
            float f[F32 ? 16 : 1];
            uint4 v[2];
            uint32_t amax;
            if constexpr (F32) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const float4 a = __builtin_bit_cast(float4, q[h]);
                    f[4 * h] = a.x;
                    f[4 * h + 1] = a.y;
                    f[4 * h + 2] = a.z;
                    f[4 * h + 3] = a.w;
                }
                const uint32_t m0 = mx_amax8(f), m1 = mx_amax8(f + 8);
                amax = m0 > m1 ? m0 : m1;
            } else {
                v[0] = q[0];
                v[1] = q[1];
                const uint32_t m0 = mx_amax8(v[0]), m1 = mx_amax8(v[1]);
                amax = m0 > m1 ? m0 : m1;
            }
            const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0xB1, 0xF, 0xF, true);
            amax = other > amax ? other : amax;
            const uint32_t s = mx_scale_byte<kE2M1>(amax);
            uint2 o;
            if constexpr (F32)
                o = make_uint2(mx_encode8_e2m1(f, amax, s), mx_encode8_e2m1(f + 8, amax, s));
            else
                o = make_uint2(mx_encode8_e2m1(v[0], amax, s), mx_encode8_e2m1(v[1], amax, s));
            if (rr < R && cc < C) {
                *reinterpret_cast<uint2*>(&row_codes[(rr * C + cc) / 8]) = o;
                if ((c16 & 1) == 0) row_scales[(rr * C + cc) / 32] = (uint8_t)s;
            }
        }
    }
}

// The same from an 8-bit checkpoint (C a multiple of 32): what unpacking it
// and packing the transpose gives, without the values in between.  A workgroup
// takes 256 rows x 128 columns, a lane 4 adjacent columns of 32 rows.
constexpr int kReCols = 128;

template <int FMT>
__global__ __launch_bounds__(kBlock) void repack_transposed_kernel(
    const uint8_t* __restrict__ ckpt, const uint8_t* __restrict__ ckpt_scales,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t R, int64_t C)
{
    __shared__ __attribute__((aligned(16))) uint8_t sC[kReCols][kTrPitch];
    __shared__ __attribute__((aligned(8))) uint8_t sS[kReCols][kTrRows / 32];
    __shared__ __attribute__((aligned(4))) uint8_t sX[kTrRows][kReCols / 32];
    const int tid = threadIdx.x;
    const int cq = tid & 31, rb = tid >> 5;   // 4 columns, row block of 32
    const int64_t r0 = (int64_t)blockIdx.x * kTrRows, c0 = (int64_t)blockIdx.y * kReCols;
    const int64_t r = r0 + 32 * rb, Cb = C / 32;
    int64_t c = c0 + 4 * cq;
    c = c < C ? c : C - 4;                    // columns past the end: loaded, not stored
    uint32_t q[32];
    if (r < R) {
#pragma unroll
        for (int i = 0; i < 32; ++i) q[i] = *reinterpret_cast<const uint32_t*>(ckpt + (r + i) * C + c);
    }
    if (r0 + tid < R) {
        const uint8_t* p = ckpt_scales + (r0 + tid) * Cb;
        if (Cb % 4 == 0) {  // one word a row (16384 x 7168: 41.7 us, by bytes 43.0)
            *reinterpret_cast<uint32_t*>(sX[tid]) = *reinterpret_cast<const uint32_t*>(p + c0 / 32);
        } else {
#pragma unroll
            for (int b = 0; b < kReCols / 32; ++b) {
                const int64_t at = c0 / 32 + b < Cb ? c0 / 32 + b : Cb - 1;
                sX[tid][b] = p[at];
            }
        }
    }
    __syncthreads();
    if (r < R) {
        uint32_t v[2][32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint2 d = mx_decode4_bf16<FMT>(q[i], mx_scale(sX[32 * rb + i][cq >> 3]));
            v[0][i] = d.x;
            v[1][i] = d.y;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            pack_column_pair(v[k], &sC[4 * cq + 2 * k][16 * rb], kTrPitch, &sS[4 * cq + 2 * k][rb], kTrRows / 32);
    }
    __syncthreads();
    store_columns<kReCols>(sC, sS, codes, scales, r0, c0, R, C);
}

// ---------------------------------------------------------------------------
// Stream mix with checkpoint.  Forward: tokens b, b + G, ... of a grid of G
// workgroups, as in the plain stream mix (the workgroups then stream a
// contiguous front of the tensors); per chunk of 8 columns the four streams
// are mixed and each is packed from the same registers.  Where a row has
// fewer than 256 chunks, 2^shift threads share a token and the workgroup
// takes several tokens at once.
// ---------------------------------------------------------------------------
constexpr int kTokensPerBlock = 16;

// out rows for one 8-column chunk: o_i = sum_j M[i][j] x_j  (M row-major 4x4)
MHC_DEV void mix_rows(const float* M, const float (*x)[8], uint4* o)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a = M[4 * i + 0] * x[0][e];
            a = __builtin_fmaf(M[4 * i + 1], x[1][e], a);
            a = __builtin_fmaf(M[4 * i + 2], x[2][e], a);
            s[e] = __builtin_fmaf(M[4 * i + 3], x[3][e], a);
        }
        o[i] = mx_pack8(s);
    }
}

// H_out may be the logits buffer itself (a lane reads its token's logits
// before it writes that token's H), so neither pointer is declared restrict.
template <int PROJ, int FMT, bool NARROW>
__global__ __launch_bounds__(kBlock) void stream_mix_ckpt_kernel(
    const uint4* __restrict__ x, const float* Hl, float* H_out, uint4* __restrict__ out,
    uint2* __restrict__ codes, uint8_t* __restrict__ scales, int64_t T, int64_t C8, int shift,
    SolverOpts o)
{
    __shared__ float sH[kTokensPerBlock][16];
    const int64_t b = blockIdx.x, G = gridDim.x;
    const int tid = threadIdx.x;
    const int64_t per = (T - b + G - 1) / G;
    const int nt = (int)(per < kTokensPerBlock ? per : kTokensPerBlock);
    if (tid < nt) {
        const int64_t t = b + G * tid;
        float a[16], h[16];
        const float4* src = reinterpret_cast<const float4*>(Hl + 16 * t);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 q = src[k];
            a[4 * k] = q.x;
            a[4 * k + 1] = q.y;
            a[4 * k + 2] = q.z;
            a[4 * k + 3] = q.w;
        }
        if (PROJ == 0) {
#pragma unroll
            for (int k = 0; k < 16; ++k) h[k] = a[k];
        } else {
            if (PROJ == 1)
                project_newton(a, h, o);
            else
                project_sinkhorn(a, h, o);
            if (H_out != nullptr) {
                float4* dst = reinterpret_cast<float4*>(H_out + 16 * t);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    dst[k] = make_float4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) sH[tid][k] = h[k];
    }
    __syncthreads();

    const int64_t Cb = (C8 + 3) / 4;  // blocks per stream row
    for (int tl = first_token<NARROW>(tid, shift); tl < nt; tl += kBlock >> shift) {
        float M[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) M[k] = sH[tl][k];
        const int64_t row = (b + G * tl) * 4;
        // the last block of a row may be part empty: its quad runs whole,
        // with zeros in the empty chunks
        for (int64_t c = tid & ((1 << shift) - 1); c < 4 * Cb; c += 1 << shift) {
            const bool in = c < C8;
            const int64_t cc = in ? c : C8 - 1;
            uint4 xin[4], oo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) xin[j] = mhc_load_stream(&x[(row + j) * C8 + cc]);
            float xf[4][8];
#pragma unroll
            for (int j = 0; j < 4; ++j) mx_unpack8(xin[j], xf[j]);
            mix_rows(M, xf, oo);
            uint32_t s[4];
            uint2 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t amax = mx_quad_max(in ? mx_amax8(xin[j]) : 0u);
                s[j] = mx_scale_byte<FMT>(amax);
                q[j] = mx_encode8<FMT>(xf[j], amax, s[j]);
            }
            if (in) {
#pragma unroll
                for (int i = 0; i < 4; ++i) mhc_store_stream(&out[(row + i) * C8 + c], oo[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) mx_store_stream(&codes[(row + j) * C8 + c], q[j]);
                if ((c & 3) == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) scales[(row + j) * Cb + (c >> 2)] = (uint8_t)s[j];
                }
            }
        }
    }
}

// Backward.  W = 64: one wave per token at a time (grid-stride); a lane
// accumulates its chunks' contribution to grad_H in 16 registers, the wave
// reduces them once per token.  W = 16, for narrow rows: 16 lanes per token.
// W = 256, for few tokens of wide rows: a workgroup per token.
template <int FMT, int W>
__global__ __launch_bounds__(kBlock) void stream_mix_bwd_ckpt_kernel(
    const uint2* __restrict__ codes, const uint8_t* __restrict__ scales,
    const float* __restrict__ H, const uint4* __restrict__ gout, uint4* __restrict__ gx,
    float* __restrict__ gH, int64_t T, int64_t C8)
{
    const int lane = threadIdx.x & (W - 1);
    const int64_t first = (int64_t)blockIdx.x * (kBlock / W) + threadIdx.x / W;
    const int64_t step = (int64_t)gridDim.x * (kBlock / W);
    const int64_t Cb = (C8 + 3) / 4;
    for (int64_t t = first; t < T; t += step) {
        float Mt[16];  // H transposed: grad_x_j = sum_i H_ij g_i
        const float4* hp = reinterpret_cast<const float4*>(H + 16 * t);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 q = hp[k];
            Mt[k] = q.x;
            Mt[4 + k] = q.y;
            Mt[8 + k] = q.z;
            Mt[12 + k] = q.w;
        }
        float acc[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] = 0.f;
        const int64_t row = t * 4;
        for (int64_t c = lane; c < C8; c += W) {
            uint4 gin[4], oo[4];
            uint2 q[4];
            uint32_t s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[j] = mx_load_stream(&codes[(row + j) * C8 + c]);
                s[j] = scales[(row + j) * Cb + (c >> 2)];
                gin[j] = mhc_load_stream(&gout[(row + j) * C8 + c]);
            }
            float gf[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) mx_unpack8(gin[i], gf[i]);
            mix_rows(Mt, gf, oo);
#pragma unroll
            for (int j = 0; j < 4; ++j) mhc_store_stream(&gx[(row + j) * C8 + c], oo[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float xf[8];
                mx_decode8<FMT>(q[j], mx_scale(s[j]), xf);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[4 * i + j] = __builtin_fmaf(gf[i][e], xf[e], acc[4 * i + j]);
            }
        }
        if constexpr (W == 256) {
            __shared__ float sP[4][16];
            const float sum = wave_sum_halving<16>(acc);
            if ((lane & 3) == 0) sP[lane >> 6][(lane & 63) >> 2] = sum;
            __syncthreads();
            if (lane < 16) gH[16 * t + lane] = (sP[0][lane] + sP[1][lane]) + (sP[2][lane] + sP[3][lane]);
            return;  // the grid has a workgroup for every token
        } else if (W == 64) {
            const float sum = wave_sum_halving<16>(acc);
            if ((lane & 3) == 0) gH[16 * t + (lane >> 2)] = sum;
        } else {
            sum16_halving<16>(acc);
            gH[16 * t + lane] = acc[0];
        }
    }
}

// Grid of the pack and unpack kernels over n chunks of the packed order.
dim3 chunk_grid(int64_t n)
{
    const int64_t per = (int64_t)kWaveChunks * (kBlock / 64);
    return dim3((unsigned)((n + per - 1) / per));
}

struct Chunks {
    int64_t n;         // chunks in the packed order
    uint32_t P8, C8;   // chunks per row there and in the unpadded rows
    bool ragged;
};

Chunks chunks_of(int64_t R, int64_t C)
{
    const int64_t Cb = (C + kMxBlock - 1) / kMxBlock;
    return Chunks{R * 4 * Cb, (uint32_t)(4 * Cb), (uint32_t)(C / 8), C % kMxBlock != 0};
}

template <int FMT, bool F32>
hipError_t pack_as(const void* x, const Packed& out, const Chunks& k, hipStream_t stream)
{
    const uint4* xv = static_cast<const uint4*>(x);
    if (k.ragged)
        hipLaunchKernelGGL((pack_kernel<FMT, F32, true>), chunk_grid(k.n), dim3(kBlock), 0, stream,
                           xv, out.codes, out.scales, nullptr, nullptr, k.n, k.P8, k.C8);
    else
        hipLaunchKernelGGL((pack_kernel<FMT, F32, false>), chunk_grid(k.n), dim3(kBlock), 0, stream,
                           xv, out.codes, out.scales, nullptr, nullptr, k.n, k.P8, k.C8);
    return hipGetLastError();
}

template <int FMT, bool F32>
hipError_t unpack_as(const Packed& in, void* x, const Chunks& k, hipStream_t stream)
{
    uint4* xv = static_cast<uint4*>(x);
    if (k.ragged)
        hipLaunchKernelGGL((unpack_kernel<FMT, F32, true>), chunk_grid(k.n), dim3(kBlock), 0,
                           stream, in.codes, in.scales, xv, k.n, k.P8, k.C8);
    else
        hipLaunchKernelGGL((unpack_kernel<FMT, F32, false>), chunk_grid(k.n), dim3(kBlock), 0,
                           stream, in.codes, in.scales, xv, k.n, k.P8, k.C8);
    return hipGetLastError();
}

template <int FMT, bool NARROW>
void mix_ckpt_as(const void* x, const float* Hl, float* H_out, void* out, const Packed& ckpt,
                 int64_t T, int64_t C, int shift, const SolverOpts* proj, hipStream_t stream)
{
    const dim3 grid(token_grid(T));
    const uint4* xv = static_cast<const uint4*>(x);
    uint4* ov = static_cast<uint4*>(out);
    uint2* cv = static_cast<uint2*>(ckpt.codes);
    if (proj == nullptr)
        hipLaunchKernelGGL((stream_mix_ckpt_kernel<0, FMT, NARROW>), grid, dim3(kBlock), 0, stream,
                           xv, Hl, nullptr, ov, cv, ckpt.scales, T, C / 8, shift, SolverOpts{});
    else if (proj->solver == 0)
        hipLaunchKernelGGL((stream_mix_ckpt_kernel<1, FMT, NARROW>), grid, dim3(kBlock), 0, stream,
                           xv, Hl, H_out, ov, cv, ckpt.scales, T, C / 8, shift, *proj);
    else
        hipLaunchKernelGGL((stream_mix_ckpt_kernel<2, FMT, NARROW>), grid, dim3(kBlock), 0, stream,
                           xv, Hl, H_out, ov, cv, ckpt.scales, T, C / 8, shift, *proj);
}

template <int FMT>
void mix_bwd_ckpt_as(const Packed& ckpt, const float* H, const void* gout, void* gx, float* gH,
                     int64_t T, int64_t C, hipStream_t stream)
{
    const uint2* cv = static_cast<const uint2*>(ckpt.codes);
    const uint4* gv = static_cast<const uint4*>(gout);
    const bool narrow = C <= 256, few = T <= 2048 && C > 512;
    const int64_t waves = narrow ? (T + 3) / 4 : T, most = waves < 8192 ? waves : 8192;
    auto* kernel = narrow ? stream_mix_bwd_ckpt_kernel<FMT, 16>
                          : (few ? stream_mix_bwd_ckpt_kernel<FMT, 256> : stream_mix_bwd_ckpt_kernel<FMT, 64>);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(few ? T : (most + 3) / 4)), dim3(kBlock), 0, stream, cv,
                       ckpt.scales, H, gv, static_cast<uint4*>(gx), gH, T, C / 8);
}

}  // namespace

hipError_t launch_ckpt_pack(const void* x, bool f32, const Packed& out, int64_t R, int64_t C,
                            int fmt, hipStream_t stream)
{
    const Chunks k = chunks_of(R, C);
    if (fmt == kE4M3)
        return f32 ? pack_as<kE4M3, true>(x, out, k, stream) : pack_as<kE4M3, false>(x, out, k, stream);
    return f32 ? pack_as<kInt8, true>(x, out, k, stream) : pack_as<kInt8, false>(x, out, k, stream);
}

hipError_t launch_ckpt_unpack(const Packed& in, void* x, bool f32, int64_t R, int64_t C, int fmt,
                              hipStream_t stream)
{
    const Chunks k = chunks_of(R, C);
    if (fmt == kE4M3)
        return f32 ? unpack_as<kE4M3, true>(in, x, k, stream) : unpack_as<kE4M3, false>(in, x, k, stream);
    return f32 ? unpack_as<kInt8, true>(in, x, k, stream) : unpack_as<kInt8, false>(in, x, k, stream);
}

hipError_t launch_mx4_quantize(const void* x, bool f32, const Packed& out, int64_t R, int64_t C,
                               bool transpose, hipStream_t stream)
{
    if (!transpose) {
        Chunks k = chunks_of(R, C);
        k.ragged = false;  // C is a multiple of 32
        const uint4* xv = static_cast<const uint4*>(x);
        if (f32)
            hipLaunchKernelGGL((pack_kernel<kE2M1, true, false>), chunk_grid(k.n), dim3(kBlock), 0,
                               stream, xv, out.codes, out.scales, nullptr, nullptr, k.n, k.P8, k.C8);
        else
            hipLaunchKernelGGL((pack_kernel<kE2M1, false, false>), chunk_grid(k.n), dim3(kBlock), 0,
                               stream, xv, out.codes, out.scales, nullptr, nullptr, k.n, k.P8, k.C8);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((R + kTrRows - 1) / kTrRows), (unsigned)((C + kTrCols - 1) / kTrCols));
    if (f32)
        hipLaunchKernelGGL((pack_transposed_kernel<true, false>), grid, dim3(kBlock), 0, stream, x,
                           static_cast<uint8_t*>(out.codes), out.scales, nullptr, nullptr, R, C);
    else
        hipLaunchKernelGGL((pack_transposed_kernel<false, false>), grid, dim3(kBlock), 0, stream, x,
                           static_cast<uint8_t*>(out.codes), out.scales, nullptr, nullptr, R, C);
    return hipGetLastError();
}

hipError_t launch_mx4_quantize_both(const void* x, bool f32, const Packed& rows, const Packed& cols,
                                    int64_t R, int64_t C, hipStream_t stream)
{
    const int64_t tiles = (R + kTrRows - 1) / kTrRows * ((C + kTrCols - 1) / kTrCols);
    auto* kernel = f32 ? pack_transposed_kernel<true, true> : pack_transposed_kernel<false, true>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(kBlock), 0, stream, x,
                       static_cast<uint8_t*>(cols.codes), cols.scales,
                       static_cast<uint32_t*>(rows.codes), rows.scales, R, C);
    return hipGetLastError();
}

hipError_t launch_mx4_quantize_ckpt(const void* x, bool f32, const Packed& out, const Packed& ckpt,
                                    int64_t R, int64_t C, int fmt, hipStream_t stream)
{
    const Chunks k = chunks_of(R, C);  // C is a multiple of 32
    auto* kernel = fmt == kE4M3
                       ? (f32 ? pack_kernel<kE4M3, true, false, true> : pack_kernel<kE4M3, false, false, true>)
                       : (f32 ? pack_kernel<kInt8, true, false, true> : pack_kernel<kInt8, false, false, true>);
    hipLaunchKernelGGL(kernel, chunk_grid(k.n), dim3(kBlock), 0, stream, static_cast<const uint4*>(x),
                       ckpt.codes, ckpt.scales, static_cast<uint32_t*>(out.codes), out.scales, k.n,
                       k.P8, k.C8);
    return hipGetLastError();
}

hipError_t launch_mx4_requantize(const Packed& ckpt, const Packed& out, int64_t R, int64_t C, int fmt,
                                 hipStream_t stream)
{
    const dim3 grid((unsigned)((R + kTrRows - 1) / kTrRows), (unsigned)((C + kReCols - 1) / kReCols));
    auto* kernel = fmt == kE4M3 ? repack_transposed_kernel<kE4M3> : repack_transposed_kernel<kInt8>;
    hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, stream, static_cast<const uint8_t*>(ckpt.codes),
                       ckpt.scales, static_cast<uint8_t*>(out.codes), out.scales, R, C);
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const Packed& in, void* x, bool f32, int64_t R, int64_t C,
                                 hipStream_t stream)
{
    Chunks k = chunks_of(R, C);
    uint4* xv = static_cast<uint4*>(x);
    if (f32)
        hipLaunchKernelGGL((unpack_kernel<kE2M1, true, false>), chunk_grid(k.n), dim3(kBlock), 0,
                           stream, in.codes, in.scales, xv, k.n, k.P8, k.C8);
    else
        hipLaunchKernelGGL((unpack_kernel<kE2M1, false, false>), chunk_grid(k.n), dim3(kBlock), 0,
                           stream, in.codes, in.scales, xv, k.n, k.P8, k.C8);
    return hipGetLastError();
}

hipError_t launch_stream_mix_ckpt(const void* x, const float* Hl, float* H_out, void* out,
                                  const Packed& ckpt, int64_t T, int64_t C, int fmt,
                                  const SolverOpts* proj, hipStream_t stream)
{
    const int shift = token_shift((C + 31) / 32 * 4);
    auto* f = fmt == kE4M3 ? (shift < 6 ? mix_ckpt_as<kE4M3, true> : mix_ckpt_as<kE4M3, false>)
                           : (shift < 6 ? mix_ckpt_as<kInt8, true> : mix_ckpt_as<kInt8, false>);
    f(x, Hl, H_out, out, ckpt, T, C, shift, proj, stream);
    return hipGetLastError();
}

hipError_t launch_stream_mix_bwd_ckpt(const Packed& ckpt, const float* H, const void* gout,
                                      void* gx, float* gH, int64_t T, int64_t C, int fmt,
                                      hipStream_t stream)
{
    if (fmt == kE4M3)
        mix_bwd_ckpt_as<kE4M3>(ckpt, H, gout, gx, gH, T, C, stream);
    else
        mix_bwd_ckpt_as<kInt8>(ckpt, H, gout, gx, gH, T, C, stream);
    return hipGetLastError();
}

}  // namespace mhc
