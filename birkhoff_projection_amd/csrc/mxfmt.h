// Blocks of 32 values that share a power-of-two scale, with 8-bit or 4-bit
// elements: the storage of activation checkpoints (e4m3, int8) and of the
// operands of the 4-bit products (e2m1).
//
// The scale byte s of a block stands for 2^(s - 127); an element stands for
// code * 2^(s - 127) (int8: code / 64).  The scale is the smallest power of
// two that keeps the block's largest magnitude inside the element type
// (448, 127/64, 6), so nothing saturates: the rule that takes the maximum's
// own exponent clips up to a quarter of the range above it, and a clipped
// outlier costs more than the half bit of resolution it saves.  Because the
// scale is a power of two, dividing by it is exact, and the one rounding of a
// value is the element's (to nearest, ties to the even code).  s is at least
// lo(), which keeps every stored value zero or a normal bf16 and fp32 number:
// 8-bit elements then convert to bf16 without any rounding.  A block with an
// infinity or a NaN has s = 255 and zero codes and reads back as NaN.
//
// A lane holds 8 consecutive values, so a block is a quad of lanes and its
// maximum takes two DPP steps.
#pragma once

#include "devmath.h"
#include "wave.h"

namespace mhc {

enum MxFormat : int { kE4M3 = 0, kInt8 = 1, kE2M1 = 2 };
constexpr int kMxBlock = 32;

typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));
typedef float mx_f32x2 __attribute__((ext_vector_type(2)));
typedef short mx_s16x2 __attribute__((ext_vector_type(2)));

MHC_DEV uint32_t mx_pack_bf16x2(float lo, float hi)
{
    mx_bf16x2 r;
    r.x = (__bf16)lo;
    r.y = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

// 8 bf16 (one uint4) <-> 8 fp32
MHC_DEV void mx_unpack8(const uint4& q, float* f)
{
    f[0] = mhc_bf16_lo(q.x);
    f[1] = mhc_bf16_hi(q.x);
    f[2] = mhc_bf16_lo(q.y);
    f[3] = mhc_bf16_hi(q.y);
    f[4] = mhc_bf16_lo(q.z);
    f[5] = mhc_bf16_hi(q.z);
    f[6] = mhc_bf16_lo(q.w);
    f[7] = mhc_bf16_hi(q.w);
}

MHC_DEV uint4 mx_pack8(const float* f)
{
    return make_uint4(mx_pack_bf16x2(f[0], f[1]), mx_pack_bf16x2(f[2], f[3]),
                      mx_pack_bf16x2(f[4], f[5]), mx_pack_bf16x2(f[6], f[7]));
}

// Bits of the largest magnitude of 8 values.  Magnitudes compare as their
// bits do, and infinities and NaNs come out largest.
MHC_DEV uint32_t mx_amax8(const float* f)
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(f[e]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    return m;
}

typedef uint16_t mx_u16x2 __attribute__((ext_vector_type(2)));

// The same from 8 packed bf16, two at a time.
MHC_DEV uint32_t mx_amax8(const uint4& q)
{
    const auto mag = [](uint32_t w) { return __builtin_bit_cast(mx_u16x2, w & 0x7fff7fffu); };
    const mx_u16x2 a = __builtin_elementwise_max(mag(q.x), mag(q.y));
    const mx_u16x2 b = __builtin_elementwise_max(mag(q.z), mag(q.w));
    const mx_u16x2 m = __builtin_elementwise_max(a, b);
    return (uint32_t)(m.x > m.y ? m.x : m.y) << 16;
}

// Maximum over the 4 lanes of a quad (all four must be active).
MHC_DEV uint32_t mx_quad_max(uint32_t v)
{
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
    v = o > v ? o : v;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
    return o > v ? o : v;
}

template <int FMT>
constexpr int mx_lo()
{
    return FMT == kE4M3 ? 10 : (FMT == kInt8 ? 7 : 2);
}

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`:
// its exponent, one more if its mantissa is above the element maximum's, less
// the element maximum's exponent.
template <int FMT>
MHC_DEV uint32_t mx_scale_byte(uint32_t amax)
{
    constexpr uint32_t kCarry = FMT == kE4M3 ? 0x1fffffu : (FMT == kInt8 ? 0x01ffffu : 0x3fffffu);
    constexpr int kExp = FMT == kE4M3 ? 8 : (FMT == kInt8 ? 0 : 2);
    int b = (int)((amax + kCarry) >> 23) - kExp;
    b = b < mx_lo<FMT>() ? mx_lo<FMT>() : b;
    b = b > 254 ? 254 : b;
    return amax >= 0x7f800000u ? 255u : (uint32_t)b;
}

// 2^(s - 127) as fp32, NaN for s = 255 (s = 0 is a subnormal).
MHC_DEV float mx_scale(uint32_t s)
{
    const uint32_t bits = s << 23;
    return __uint_as_float(s == 255u ? 0x7fc00000u : (s == 0u ? 0x00400000u : bits));
}

MHC_DEV uint32_t mx_perm(uint32_t hi, uint32_t lo, uint32_t sel)
{
    return __builtin_amdgcn_perm(hi, lo, sel);
}

// Largest magnitude that reads back finite: the next element would stand for
// 2^128.  Only a block whose maximum is above it looks at its values.
template <int FMT>
MHC_DEV constexpr uint32_t mx_limit()
{
    return FMT == kE4M3 ? 0x7f700000u : (FMT == kInt8 ? 0x7f7e0000u : 0x7f400000u);
}

template <int FMT>
MHC_DEV void mx_limit8(float* f, uint32_t amax)
{
    if (amax > mx_limit<FMT>()) {
        const float top = __uint_as_float(mx_limit<FMT>());
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = mhc_max(mhc_min(f[e], top), -top);
    }
}

// 8 values to 8 codes of one byte (codes of a block with s = 255: see
// mx_encode8).
MHC_DEV uint2 mx_encode8_e4m3(const float* f, uint32_t s)
{
    // the conversion divides by the scale operand's power of two
    const float sc = mx_scale(s);
    mx_s16x2 a = {0, 0}, b = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, f[0], f[1], sc, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, f[2], f[3], sc, true);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, f[4], f[5], sc, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, f[6], f[7], sc, true);
    return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}

MHC_DEV uint2 mx_encode8_int8(const float* f, uint32_t s)
{
    // v * 64 / 2^(s-127) is exact; adding 1.5 * 2^23 rounds it to an integer
    // (nearest even) held in the low mantissa bits, whose low byte is the
    // two's complement code.
    const float k = __uint_as_float((260u - s) << 23);
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__builtin_fmaf(f[e], k, 12582912.f));
    const auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        return mx_perm(mx_perm(d, c, 0x0c0c0400u), mx_perm(b, a, 0x0c0c0400u), 0x05040100u);
    };
    return make_uint2(four(w[0], w[1], w[2], w[3]), four(w[4], w[5], w[6], w[7]));
}

// amax: bits of the largest magnitude of the block, s: its scale byte.  Values
// above mx_limit are stored as that; f is changed then.
template <int FMT>
MHC_DEV uint2 mx_encode8(float* f, uint32_t amax, uint32_t s)
{
    mx_limit8<FMT>(f, amax);
    const uint2 c = FMT == kE4M3 ? mx_encode8_e4m3(f, s) : mx_encode8_int8(f, s);
    return s == 255u ? make_uint2(0u, 0u) : c;
}

// 8 values to 8 codes of 4 bits, the first in the low half of the first byte.
MHC_DEV uint32_t mx_encode8_e2m1(float* f, uint32_t amax, uint32_t s)
{
    mx_limit8<kE2M1>(f, amax);
    const float sc = mx_scale(s);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0], f[1], sc, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2], f[3], sc, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4], f[5], sc, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6], f[7], sc, 3);
    return s == 255u ? 0u : r;
}

MHC_DEV uint32_t mx_encode8_e2m1(const uint4& q, uint32_t amax, uint32_t s)
{
    if (amax > mx_limit<kE2M1>()) {
        float f[8];
        mx_unpack8(q, f);
        return mx_encode8_e2m1(f, amax, s);
    }
    const float sc = mx_scale(s);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf16x2, q.x), sc, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf16x2, q.y), sc, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf16x2, q.z), sc, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf16x2, q.w), sc, 3);
    return s == 255u ? 0u : r;
}

// 4 codes of one byte (a word) to 4 fp32 values.  Exact.
template <int FMT>
MHC_DEV void mx_decode4(uint32_t w, float sc, float* f)
{
    if (FMT == kE4M3) {
        const mx_f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, sc, false);
        const mx_f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, sc, true);
        f[0] = a.x;
        f[1] = a.y;
        f[2] = b.x;
        f[3] = b.y;
    } else {
        const float k = sc * 0.015625f;
        f[0] = (float)(int8_t)w * k;
        f[1] = (float)(int8_t)(w >> 8) * k;
        f[2] = (float)(int8_t)(w >> 16) * k;
        f[3] = (float)(int8_t)(w >> 24) * k;
    }
}

template <int FMT>
MHC_DEV void mx_decode8(const uint2& c, float sc, float* f)
{
    mx_decode4<FMT>(c.x, sc, f);
    mx_decode4<FMT>(c.y, sc, f + 4);
}

// 4 codes of one byte to 4 bf16 (two words).  Exact: a stored value has at
// most 8 significant bits and is a normal bf16.
template <int FMT>
MHC_DEV uint2 mx_decode4_bf16(uint32_t w, float sc)
{
    if (FMT == kE4M3) {
        const mx_bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, false);
        const mx_bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, true);
        return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    }
    float f[4];
    mx_decode4<FMT>(w, sc, f);
    return make_uint2(mx_pack_bf16x2(f[0], f[1]), mx_pack_bf16x2(f[2], f[3]));
}

// 8 codes of 4 bits to 8 fp32 values.  Exact.
MHC_DEV void mx_decode8_e2m1(uint32_t w, float sc, float* f)
{
    const mx_f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 0);
    const mx_f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 1);
    const mx_f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 2);
    const mx_f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 3);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
    f[4] = c.x;
    f[5] = c.y;
    f[6] = d.x;
    f[7] = d.y;
}

// Streaming 8-byte accesses (data moved once).
typedef unsigned int mx_u32x2 __attribute__((ext_vector_type(2)));
MHC_DEV uint2 mx_load_stream(const uint2* p)
{
    const mx_u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const mx_u32x2*>(p));
    return make_uint2(v.x, v.y);
}
MHC_DEV void mx_store_stream(uint2* p, const uint2& q)
{
    const mx_u32x2 v = {q.x, q.y};
    __builtin_nontemporal_store(v, reinterpret_cast<mx_u32x2*>(p));
}

// Sums over each 16 lanes of a wave of N = 16 or 32 partials: lane l holds
// those of partials (N / 16) (l % 16) + 0 .. N / 16 - 1 in v[0 .. N / 16 - 1].
template <int N>
MHC_DEV void sum16_halving(float* v)
{
    halve_dpp<kDppBit3, 3, N / 2>(v);
    halve_dpp<kDppBit2, 2, N / 4>(v);
    halve_dpp<kDppBit1, 1, N / 8>(v);
    halve_dpp<kDppBit0, 0, N / 16>(v);
}

// A token's place for a thread of a workgroup in which 2^shift share a token.
// From 64 on a wave is within one token, whose rows then have scalar bases;
// below that, NARROW kernels keep the addresses per lane.
template <bool NARROW>
MHC_DEV int first_token(int tid, int shift)
{
    return NARROW ? tid >> shift : __builtin_amdgcn_readfirstlane(tid >> shift);
}

// log2 of the threads of a workgroup that share a token of `chunks` chunks:
// the fewest that take the row in one go, at least a quad (a block).
inline int token_shift(int64_t chunks)
{
    int shift = 2;
    while (shift < 8 && (1 << shift) < chunks) ++shift;
    return shift;
}

}  // namespace mhc
