// Products of MXFP4 matrices (mxfmt.h, e2m1) on the scaled matrix
// instructions of gfx950:  y[m,n] = sum_k a[m,k] b[n,k].
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 by 64 x 32 elements and
// applies both operands' block scales in the same instruction: lane l holds
// the 32 elements (16 bytes) of row l % 32, block l / 32, and one byte of a
// register as that block's scale.  Products of two e2m1 elements are exact,
// the accumulation is fp32.
#include <type_traits>

#include "ldscopy.h"
#include "mxfmt.h"
#include "qkernels.h"

namespace mhc {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // operand type code of the scaled matrix instructions

MHC_DEV i32x8 frag(const uint4& q)
{
    return i32x8{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
}

// What becomes of a product: y stored as bf16 or fp32, or the layer's
// write-back x_out[t,i,:] = H_post[t,i] y[t,:] + sum_j H_res[t,i,j] x[t,j,:]
// (y itself stored only if `out` is given).
enum Epilogue : int { kStoreBf16 = 0, kStoreF32 = 1, kWriteBack = 2 };

struct Mx4Args {
    const uint8_t* a;   // [M, K/2] codes (or, fused, the values of a)
    const uint8_t* as;  // [M, K/32]
    const uint8_t* b;   // [N, K/2]
    const uint8_t* bs;  // [N, K/32]
    void* out;          // [M, N]
    const uint4* x;     // write-back: [M, 4, N] bf16
    const float* Hpost; // [M, 4]
    const float* Hres;  // [M, 4, 4]
    uint4* x_out;       // [M, 4, N] bf16
    int64_t M, N, K;
};

// x_out of 8 columns (chunk c) of row m from y and the four streams xq;
// h: H_post[0..3], then H_res row by row.
MHC_DEV void write_back8(const Mx4Args& p, int64_t m, int64_t c, const float* y, const uint4 (&xq)[4],
                         const float4 (&h)[5])
{
    const int64_t N8 = p.N / 8;
    if (p.out != nullptr) reinterpret_cast<uint4*>(p.out)[m * N8 + c] = mx_pack8(y);
    const float post[4] = {h[0].x, h[0].y, h[0].z, h[0].w};
    float xs[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) mx_unpack8(xq[j], xs[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float s = post[i] * y[e];
            s = __builtin_fmaf(h[1 + i].x, xs[0][e], s);
            s = __builtin_fmaf(h[1 + i].y, xs[1][e], s);
            s = __builtin_fmaf(h[1 + i].z, xs[2][e], s);
            o[e] = __builtin_fmaf(h[1 + i].w, xs[3][e], s);
        }
        mhc_store_stream(&p.x_out[(m * 4 + i) * N8 + c], mx_pack8(o));
    }
}

// Part q of a row's maps: 0 H_post, 1..4 the rows of H_res.
MHC_DEV float4 map_part(const Mx4Args& p, int64_t m, int q)
{
    return q == 0 ? reinterpret_cast<const float4*>(p.Hpost)[m]
                  : reinterpret_cast<const float4*>(p.Hres)[4 * m + q - 1];
}

MHC_DEV void load_x8(const Mx4Args& p, int64_t m, int64_t c, uint4 (&xq)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) xq[j] = mhc_load_stream(&p.x[(m * 4 + j) * (p.N / 8) + c]);
}

// 8 consecutive columns (n a multiple of 8) of row m of the product.
template <int EPI>
MHC_DEV void store8(const Mx4Args& p, int64_t m, int64_t n, const float* y)
{
    if (EPI == kStoreF32) {
        float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + m * p.N + n);
        o[0] = make_float4(y[0], y[1], y[2], y[3]);
        o[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
        reinterpret_cast<uint4*>(p.out)[m * (p.N / 8) + n / 8] = mx_pack8(y);
    }
}

// ---------------------------------------------------------------------------
// Tiled product.  Workgroup: WM x WN waves, each 32 TM x 32 TN outputs, K in
// stages of 256, 4 steps of 64: 128 bytes of codes and 8 scale bytes per row.
//
// LDS: NBUF stage buffers.  A row is 8 pieces of 16 bytes, piece c of row r at
// place c ^ (r / 2 % 8): the 16 rows that one phase of a read covers then fall
// on all 64 banks.  Each 4 scale bytes of a row are one word; a lane of block
// half h = lane / 32 shifts it by 8 h and finds the scales of two steps in
// bytes 0 and 2, which the instruction selects.
//
// Pipeline: copies run NBUF - 1 stages ahead, straight from global memory to
// LDS, and two register sets hold fragments: while one step multiplies, the
// next one's are read.  A stage's last fragments are in registers before its
// last step, so the one barrier per stage stands there: behind it the next
// stage's first fragments are read and the copies of the stage NBUF ahead go
// into the freed buffer, between that step's products.  The barrier waits for
// the next stage's copies only (the counter retires in order).
//
// Scales.  A row's scale bytes lie K / 32 apart from the next row's, so every
// lane of a copy fetches from a line of its own, however little it takes: with
// a word per lane, two words of each row a stage, the scales cost as many line
// look-ups as the codes (8192 x 8192 x 4096 in tiles of 256 155 us, of 128 244;
// with the same words from one line, a test, 138 and 195).  Where K is a
// multiple of 512 (kPairs) a lane takes the 16 bytes of two stages at once, a
// quarter of the look-ups.  kWordwise: K is another multiple of 256.
//
// kTail: K is no multiple of 256.  The last stage's pieces past K repeat the
// row's last piece; scale bytes of 0 in both operands make them 2^-254 times
// their product of at most 32 * 36, which is nothing to a sum in 32 bits.
// Rows of scales may then start at any byte: the aligned words around a row's
// bytes are copied, one more than it has, and a lane shifts its bytes out of
// two of them.
// ---------------------------------------------------------------------------

constexpr int kStageK = 256;                  // of K in a stage
constexpr int kRowBytes = kStageK / 2;        // codes of a row there
constexpr int kRowBlocks = kStageK / 32;      // and its scale bytes
constexpr int kWords = kRowBlocks / 4;

template <int TM, int TN>
struct Frags {
    uint4 a[TM], b[TN];
};

// place of piece c of row r
MHC_DEV int piece_at(int r, int c)
{
    return c ^ ((r >> 1) & 7);
}

template <int S, int TM, int TN>
MHC_DEV void read_frags(Frags<TM, TN>& f, const uint8_t* sA, const uint8_t* sB, int ra, int rb,
                        int kh)
{
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = ra + 32 * i;
        f.a[i] = *reinterpret_cast<const uint4*>(sA + r * kRowBytes + 16 * piece_at(r, 2 * S + kh));
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int r = rb + 32 * j;
        f.b[j] = *reinterpret_cast<const uint4*>(sB + r * kRowBytes + 16 * piece_at(r, 2 * S + kh));
    }
}

// scale words of a stage: [word][tile]
template <int W, int TM, int TN>
struct Scales {
    uint32_t a[W][TM], b[W][TN];
};

template <int S, int W, int TM, int TN>
MHC_DEV void mma_one(const Frags<TM, TN>& f, const Scales<W, TM, TN>& x, f32x16 (&acc)[TM][TN], int i,
                     int j)
{
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        frag(f.a[i]), frag(f.b[j]), acc[i][j], kFp4, kFp4, 2 * (S & 1), (int)x.a[S / 2][i], 2 * (S & 1),
        (int)x.b[S / 2][j]);
}

template <int S, int W, int TM, int TN>
MHC_DEV void mma_step(const Frags<TM, TN>& f, const Scales<W, TM, TN>& x, f32x16 (&acc)[TM][TN])
{
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < TM * TN; ++q) mma_one<S>(f, x, acc, q / TN, q % TN);
    __builtin_amdgcn_sched_barrier(0);
}

enum Mx4Scales : int { kPairs = 0, kWordwise = 1, kTail = 2 };

template <int TM, int TN, int WM, int WN, int NBUF, int EPI, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void mx4_tile_kernel(Mx4Args p, unsigned gm, unsigned gn)
{
    constexpr bool TAIL = MODE == kTail, PAIRS = MODE == kPairs;
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, ROWS = BM + BN;
    constexpr int kCopied = TAIL ? kWords + 1 : kWords;  // scale words of a row
    constexpr int kBlock = 64 * WM * WN;
    constexpr int kBytes = ROWS * kRowBytes;       // codes of one stage
    constexpr int TS = TN < 2 ? TN : 2;            // tiles side by side in an output strip
    constexpr int kPitch = 32 * TS + 4;            // floats per row of a strip
    static_assert(WM * WN * 32 * kPitch * 4 + BM * 80 <= NBUF * kBytes,
                  "output strips and maps fit the stage buffers");
    __shared__ __attribute__((aligned(16))) uint8_t sC[NBUF][kBytes];
    __shared__ uint32_t sX[PAIRS ? 1 : NBUF][PAIRS ? 1 : kCopied][PAIRS ? 1 : ROWS];
    __shared__ uint4 sP[2][PAIRS ? ROWS : 1];      // a row's scales of two stages
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // Workgroups go to the 8 dies in turn; each die takes a run of
    // consecutive tiles, in bands of 4 tile rows, so that the rows and columns
    // its workgroups share stay in its cache.
    unsigned tm, tn;
    {
        const unsigned total = gm * gn, id = blockIdx.x;
        const unsigned per = total / 8, extra = total % 8, die = id % 8;
        unsigned t = die * per + (die < extra ? die : extra) + id / 8;
        const unsigned band = t / (4 * gn), rows = gm - 4 * band < 4 ? gm - 4 * band : 4;
        t -= 4 * gn * band;
        // (divisions run on the vector unit; the tile is the wave's own again)
        tm = __builtin_amdgcn_readfirstlane(4 * band + t % rows);
        tn = __builtin_amdgcn_readfirstlane(t / rows);
    }
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int64_t Kb = p.K / 2, Ks = p.K / 32;
    const int wm = w % WM, wn = w / WM;
    const int ra = 32 * TM * wm + (lane & 31), rb = 32 * TN * wn + (lane & 31);
    const int kh = lane >> 5;
    const int stages = (int)((p.K + kStageK - 1) / kStageK);

    // A thread copies piece c of every kStep-th row from tid / 8 on (c and
    // its place in LDS are fixed by tid).  Rows past the matrix repeat its
    // last one; their products are not used.  Row offsets fit 32 bits: 255
    // rows of at most 2^23 bytes.
    constexpr int kStep = kBlock / 8;
    constexpr int NA = BM / kStep, NB = BN / kStep;     // code copies per thread and stage
    constexpr int NX = (ROWS + kBlock - 1) / kBlock;    // scale copies
    static_assert(BM % kStep == 0 && BN % kStep == 0 && kStep % 16 == 0, "whole copies, one swizzle per thread");
    const int row0 = tid / 8, c16 = 16 * piece_at(row0, tid % 8);
    const uint8_t* baseA = p.a + m0 * Kb;
    const uint8_t* baseB = p.b + n0 * Kb;
    uint32_t offA[NA], offB[NB];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int64_t r = kStep * i + row0, last = p.M - 1 - m0;
        offA[i] = (uint32_t)((r < last ? r : last) * Kb) + c16;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t r = kStep * i + row0, last = p.N - 1 - n0;
        offB[i] = (uint32_t)((r < last ? r : last) * Kb) + c16;
    }
    // Scale words: a wave's 64 rows all belong to A or all to B (BM and BN are
    // multiples of 64).  Where the rows are no multiple of the threads, some
    // waves copy rows again that others copy too.
    static_assert(BM % 64 == 0 && BN % 64 == 0, "a wave's scale rows are one matrix's");
    uint32_t offX[NX], endX[NX];  // endX: offset of the matrix's last word of scales
    const uint8_t* baseX[NX];
    int rowX[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int first = (64 * w + kBlock * i) % ROWS;  // wave-uniform
        const bool isA = first < BM;
        const int64_t b0 = isA ? m0 : n0, n = isA ? p.M : p.N, base = (b0 * Ks) & ~(int64_t)3;
        const int64_t r = b0 + first - (isA ? 0 : BM) + lane;
        baseX[i] = (isA ? p.as : p.bs) + base;
        offX[i] = (uint32_t)((((r < n ? r : n - 1) * Ks) & ~(int64_t)3) - base);
        const int64_t end = ((n * Ks - 1) & ~(int64_t)3) - base;
        endX[i] = (uint32_t)(end < 0xffffffff ? end : 0xffffffff);
        rowX[i] = first;
    }
    // byte of its first word where a lane's scales begin (the same for all its
    // rows: they are 32 apart)
    const uint32_t sa = TAIL ? (uint32_t)((m0 + ra) * Ks) & 3 : 0;
    const uint32_t sb = TAIL ? (uint32_t)((n0 + rb) * Ks) & 3 : 0;
    // TAIL, last stage: bytes a thread's piece is past the row, and the lane's
    // scale bytes (0 and 2 of each word) that exist
    uint32_t cutLast = 0, maskLast[kWords];
    if (TAIL) {
        const int64_t over = (int64_t)(stages - 1) * kRowBytes + c16 - (Kb - 16);
        cutLast = over > 0 ? (uint32_t)over : 0u;
        const int64_t left = Ks - kRowBlocks * (int64_t)(stages - 1) - kh;
#pragma unroll
        for (int q = 0; q < kWords; ++q)
            maskLast[q] = (left > 4 * q ? 0xffu : 0u) | (left > 4 * q + 2 ? 0xff0000u : 0u);
    }
    const uint32_t ldsC = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&sC[0][0];
    const uint32_t ldsX = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint32_t*)&sX[0][0];
    constexpr int NC = NA + NB + (PAIRS ? 0 : kCopied * NX);  // copies per thread and stage
    const uint32_t ldsP = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint4*)&sP[0][0];
    // kPairs: scales of stages st and st + 1 (st even) to the pair's buffer
    const auto copy_pair = [&](int st, int pair, int x) {
        copy16_to_lds(baseX[x], offX[x] + (uint32_t)st * kRowBlocks, ldsP + 16 * ((pair & 1) * ROWS + rowX[x]));
    };
    const auto copy = [&](int st, int buf, int i) {  // copy i of stage st
        if (i < NA + NB) {
            const uint32_t cut = TAIL && st == stages - 1 ? cutLast : 0u;
            const bool isA = i < NA;
            const uint8_t* base = (isA ? baseA : baseB) + (int64_t)st * kRowBytes;
            copy16_to_lds(base, (isA ? offA[isA ? i : 0] : offB[isA ? 0 : i - NA]) - cut,
                          ldsC + buf * kBytes + 16 * (kBlock * i + 64 * w));
        } else {
            const int x = (i - NA - NB) / kCopied, q = (i - NA - NB) % kCopied;
            const uint32_t at = (uint32_t)st * kRowBlocks + 4 * q;  // at most 2^19
            uint32_t off = offX[x] + at;
            if (TAIL) off = off < endX[x] ? off : endX[x];  // a word past the last: not used
            copy4_to_lds(baseX[x], off, ldsX + 4 * ((buf * kCopied + q) * ROWS + rowX[x]));
        }
    };
    // Stages past the last one repeat it and nothing uses them: the loop stays
    // one block, which keeps the products between the copies (the compiler
    // sinks them past a branch, and then nothing overlaps).
    const auto clamped = [&](int st) { return st < stages ? st : stages - 1; };
    const auto scales = [&](Scales<kCopied, TM, TN>& y, int buf, int st) {
        if constexpr (PAIRS) {
            const auto two = [&](int row) {
                return *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(&sP[(st >> 1) & 1][row]) +
                                                       8 * (st & 1));
            };
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const uint2 v = two(ra + 32 * i);
                y.a[0][i] = v.x;
                y.a[1][i] = v.y;
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const uint2 v = two(BM + rb + 32 * j);
                y.b[0][j] = v.x;
                y.b[1][j] = v.y;
            }
            return;
        }
#pragma unroll
        for (int q = 0; q < kCopied; ++q) {
#pragma unroll
            for (int i = 0; i < TM; ++i) y.a[q][i] = sX[buf][q][ra + 32 * i];
#pragma unroll
            for (int j = 0; j < TN; ++j) y.b[q][j] = sX[buf][q][BM + rb + 32 * j];
        }
    };
    // the lane's own scales in bytes 0 and 2
    const auto shifted = [&](Scales<kWords, TM, TN>& x, const Scales<kCopied, TM, TN>& y, int st) {
        uint32_t mask = 0;
        const auto pick = [&](uint32_t lo, uint32_t hi, uint32_t s) {
            if (!TAIL) return lo >> (8 * kh);
            return (__builtin_amdgcn_alignbyte(hi, lo, s) >> (8 * kh)) & mask;
        };
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
            constexpr int one = TAIL ? 1 : 0;
            if (TAIL) mask = st == stages - 1 ? maskLast[q] : 0xff00ffu;
#pragma unroll
            for (int i = 0; i < TM; ++i) x.a[q][i] = pick(y.a[q][i], y.a[q + one][i], sa);
#pragma unroll
            for (int j = 0; j < TN; ++j) x.b[q][j] = pick(y.b[q][j], y.b[q + one][j], sb);
        }
    };
    // next stage's copies landed, everybody's reads of this one done (a stage
    // that copies a pair's scales too waits for that much more)
    const auto hand_over = [&]() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"((NBUF - 2) * NC) : "memory");
    };
    static_assert((NBUF - 2) * NC < 64, "the copies in flight fit the counter");

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    Frags<TM, TN> f0, f1;
    Scales<kWords, TM, TN> x;
    Scales<kCopied, TM, TN> y;
#pragma unroll
    for (int b = 0; b < NBUF; ++b) {
        if (b == NBUF - 1) hand_over();  // stage 0 (NBUF - 1 stages are on their way)
#pragma unroll
        for (int i = 0; i < NC; ++i) copy(clamped(b), b, i);
        if constexpr (PAIRS) {
            if (b % 2 == 0) {
#pragma unroll
                for (int x = 0; x < NX; ++x) copy_pair(clamped(b) & ~1, b / 2, x);
            }
        }
    }
    scales(y, 0, 0);
    shifted(x, y, 0);
    read_frags<0>(f0, sC[0], sC[0] + BM * kRowBytes, ra, rb, kh);
    int buf = 0;
    const auto stage = [&](int st, auto odd) {
        constexpr bool kPair = PAIRS && (odd.value + NBUF) % 2 == 0;  // stage st + NBUF begins a pair
        constexpr int kAll = NC + (kPair ? NX : 0);
        const uint8_t* cA = sC[buf];
        const uint8_t* cB = cA + BM * kRowBytes;
        const int nxt = buf + 1 < NBUF ? buf + 1 : 0;
        read_frags<1>(f1, cA, cB, ra, rb, kh);
        mma_step<0>(f0, x, acc);
        read_frags<2>(f0, cA, cB, ra, rb, kh);
        mma_step<1>(f1, x, acc);
        read_frags<3>(f1, cA, cB, ra, rb, kh);
        mma_step<2>(f0, x, acc);
        hand_over();
        const uint8_t* nA = sC[nxt];
        scales(y, nxt, st + 1);
        read_frags<0>(f0, nA, nA + BM * kRowBytes, ra, rb, kh);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int kPer = (kAll + TM * TN - 1) / (TM * TN);  // copies behind each product
#pragma unroll
        for (int q = 0; q < TM * TN; ++q) {
            mma_one<3>(f1, x, acc, q / TN, q % TN);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = kPer * q; i < kPer * (q + 1) && i < kAll; ++i) {
                if (i < NC) copy(clamped(st + NBUF), buf, i);
                else copy_pair(clamped(st + NBUF) & ~1, (st + NBUF) / 2, i - NC);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        shifted(x, y, st + 1);
        buf = nxt;
    };
    if constexpr (PAIRS) {
        for (int st = 0; st < stages; st += 2) {  // K is a multiple of 512
            stage(st, std::integral_constant<int, 0>{});
            stage(st + 1, std::integral_constant<int, 1>{});
        }
    } else {
        for (int st = 0; st < stages; ++st) stage(st, std::integral_constant<int, 0>{});
    }
    // every wave is done with the stage buffers before they hold the outputs
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    // D: column lane % 32, rows (v % 4) + 8 (v / 4) + 4 (lane / 32).  Strips of
    // 32 rows go through the wave's own LDS to 8 columns per lane.  The
    // write-back is bound by the memory behind it: the tile's maps are put in
    // LDS first, and a strip's x is all under way before the strip is written.
    float* strip = reinterpret_cast<float*>(&sC[0][0]) + w * 32 * kPitch;
    float4* maps = reinterpret_cast<float4*>(&sC[0][0] + WM * WN * 32 * kPitch * 4);  // [BM][5]
    if constexpr (EPI == kWriteBack) {
        for (int e = tid; e < BM * 5; e += kBlock) {
            const int64_t m = m0 + e / 5;
            maps[e] = map_part(p, m < p.M ? m : p.M - 1, e % 5);
        }
        __syncthreads();
    }
    constexpr int kLanes = 4 * TS;                 // lanes per row
    constexpr int kQ = 32 * kLanes / 64;           // rows of a strip per lane
    const int64_t mw = m0 + 32 * TM * wm, nw = n0 + 32 * TN * wn;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int jj = 0; jj < TN; jj += TS) {
            const int r0 = lane / kLanes, c = 8 * (lane % kLanes);
            const int64_t n = nw + 32 * jj + c;
            uint4 xq[kQ][4];
            if constexpr (EPI == kWriteBack) {
#pragma unroll
                for (int q = 0; q < kQ; ++q) {
                    const int64_t m = mw + 32 * i + (64 / kLanes) * q + r0;
                    load_x8(p, m < p.M ? m : p.M - 1, (n < p.N ? n : p.N - 8) / 8, xq[q]);
                }
            }
            mhc_wave_lds_fence();  // the previous strip's reads come first
#pragma unroll
            for (int j = 0; j < TS; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    strip[((v & 3) + 8 * (v >> 2) + 4 * kh) * kPitch + 32 * j + (lane & 31)] = acc[i][jj + j][v];
            mhc_wave_lds_fence();
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                const int r = (64 / kLanes) * q + r0;
                const int64_t m = mw + 32 * i + r;
                if (m < p.M && n < p.N) {
                    const float4 y0 = *reinterpret_cast<const float4*>(&strip[r * kPitch + c]);
                    const float4 y1 = *reinterpret_cast<const float4*>(&strip[r * kPitch + c + 4]);
                    const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
                    if constexpr (EPI == kWriteBack) {
                        const float4* h = maps + 5 * (m - m0);
                        write_back8(p, m, n / 8, y, xq[q], {h[0], h[1], h[2], h[3], h[4]});
                    } else {
                        store8<EPI>(p, m, n, y);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows of a: bound by reading b once.  A workgroup takes 16 rows of b and
// 16 of a (all of them, mostly), K in panels of up to PT tiles of 256.  Waves 4..7
// copy the panel of b to LDS, every instruction 8 whole lines of 128 bytes;
// meanwhile waves 0..3 put a there.  Then the 8 waves share the tiles; their
// partial sums meet in LDS at the end and are added in wave order.
//
// Whole lines are the point: loading b in the layout the instruction wants (16
// bytes of 64 different lines at a time) ran at a third of this speed.
//
// SRC 0: a is packed and copied like b.  SRC 1, 2: a is bf16 or fp32, and every
// workgroup quantises it for itself while its copies of b are under way: one
// launch instead of two, for a call that lasts a few microseconds.
//
// LDS per tile: 16 rows of b, then MR rows of a (MR: M rounded up to a power of
// two), each 128 bytes with piece c of row r at place c ^ (r / 2 % 8); then 8 scale
// bytes of each row.  Lanes of rows past M use row M - 1; only their own
// columns of the result, which are dropped, depend on them.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;

struct FewShape {
    int MR, LR, PT;      // rows of a in LDS and their logarithm, tiles per panel
    unsigned groups;     // of 16 rows of a
    unsigned lds;        // bytes
};

__host__ __device__ constexpr int few_tile_bytes(int MR) { return (16 + MR) * 136; }

template <int SRC, int EPI>
__global__ __launch_bounds__(kFewThreads) void mx4_few_kernel(Mx4Args p, FewShape sh)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
    __shared__ float sR[kFewWaves][16][17];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = lane & 15, kq = lane >> 4;
    // workgroups b, b + 8, ... run on one die: there the row groups of a
    // follow each other on the same rows of b
    const unsigned q8 = blockIdx.x / 8;
    const int64_t n0 = (int64_t)(q8 / sh.groups * 8 + blockIdx.x % 8) * 16;
    const int64_t m0 = (int64_t)(q8 % sh.groups) * 16;
    if (n0 >= p.N) return;
    const int M = (int)(p.M - m0 < 16 ? p.M - m0 : 16), MR = sh.MR, PT = sh.PT;
    const int64_t Ks = p.K / 32, Kb = p.K / 2;
    const int tiles = (int)((p.K + 255) / 256);
    const bool words = (Ks & 3) == 0;  // scale rows are whole words
    uint8_t* sB = sm;                                  // [PT][16][128]
    uint8_t* sA = sB + (int64_t)PT * 16 * 128;         // [PT][MR][128]
    uint8_t* xB = sA + (int64_t)PT * MR * 128;         // [PT][16][8]
    uint8_t* xA = xB + PT * 16 * 8;                    // [PT][MR][8]
    const auto lds_at = [](const void* q) {
        return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)q);
    };
    const int nB = (int)(p.N - n0 < 16 ? p.N - n0 : 16);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const int ma = row < M ? row : M - 1;

    // codes of 2^lr rows (`have` exist) of a panel to LDS: 4 waves, 8 rows of
    // 128 bytes per instruction (lanes past the end are switched off)
    const auto copy_codes = [&](const uint8_t* src, int lr, int have, int t0, int nt, uint8_t* dst, int wv) {
        const uint32_t l0 = lds_at(dst);
        const int pieces = (nt << lr) * 8;
        for (int q = 64 * wv; q < pieces; q += 256) {
            const int e = q + lane;
            if (e < pieces) {
                const int r = (e >> 3) & ((1 << lr) - 1), t = e >> (3 + lr), c = (e & 7) ^ ((r >> 1) & 7);
                int64_t kb = (int64_t)(t0 + t) * 128 + 16 * c;
                kb = kb < Kb ? kb : Kb - 16;  // bytes past the row: not used
                const int64_t rr = r < have ? r : have - 1;
                copy16_to_lds(src, (uint32_t)(rr * Kb + kb), l0 + 16 * q);
            }
        }
    };
    const auto copy_scales = [&](const uint8_t* src, int lr, int have, int t0, int nt, uint8_t* dst, int wv) {
        const uint32_t l0 = lds_at(dst);
        const int n = (nt << lr) * 2;
        for (int q = 64 * wv; q < n; q += 256) {
            const int e = q + lane;
            if (e < n) {
                const int r = (e >> 1) & ((1 << lr) - 1), t = e >> (1 + lr);
                int64_t ks = (int64_t)(t0 + t) * 8 + 4 * (e & 1);
                const int64_t rr = r < have ? r : have - 1;
                if (words) {
                    ks = ks < Ks ? ks : Ks - 4;
                    copy4_to_lds(src, (uint32_t)(rr * Ks + ks), l0 + 4 * q);
                } else {
                    uint32_t v = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v |= (uint32_t)(ks + k < Ks ? src[rr * Ks + ks + k] : 127) << (8 * k);
                    reinterpret_cast<uint32_t*>(dst)[e] = v;
                }
            }
        }
    };

    for (int t0 = 0; t0 < tiles; t0 += PT) {
        const int nt = tiles - t0 < PT ? tiles - t0 : PT;
        if (t0 > 0) {  // everybody is done with the panel before
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        // quantising: 8 columns per lane, a block per quad, 4 chunks' loads at
        // once; all counts are multiples of 4, so a quad of lanes is whole
        const int C8 = (int)(p.K / 8), c0 = t0 * 32;
        const int nc = C8 - c0 < nt * 32 ? C8 - c0 : nt * 32;  // chunks per row
        const int total = M * nc;
        uint4 v[4][SRC > 0 ? SRC : 1];
        int mi[4], ii[4];
        const auto load_a = [&](int j) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int e = j + 256 * u < total ? j + 256 * u : total - 1;
                mi[u] = M == 1 ? 0 : e / nc;
                ii[u] = e - mi[u] * nc;
                const int64_t g = (int64_t)mi[u] * C8 + c0 + ii[u];
#pragma unroll
                for (int h = 0; h < SRC; ++h) v[u][h] = reinterpret_cast<const uint4*>(p.a)[SRC * g + h];
            }
        };
        if constexpr (SRC > 0) {
            // Returns come in order: behind the copies of b, a would arrive
            // last and its quantisation stand alone at the end (9.9 us instead
            // of 6.5 for 1 x 7168 x 7168).  So its first loads go out before.
            if (w < 4) load_a(tid);
            asm volatile("s_barrier" ::: "memory");
        }
        if (w >= 4) {
            copy_codes(p.b + n0 * Kb, 4, nB, t0, nt, sB, w - 4);
            copy_scales(p.bs + n0 * Ks, 4, nB, t0, nt, xB, w - 4);
        } else if constexpr (SRC == 0) {
            copy_codes(p.a + m0 * Kb, sh.LR, M, t0, nt, sA, w);
            copy_scales(p.as + m0 * Ks, sh.LR, M, t0, nt, xA, w);
        } else {
            for (int j = tid; j < total; j += 1024) {
                if (j != tid) load_a(j);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (j + 256 * u >= total) break;
                    uint32_t code, s;
                    if constexpr (SRC == 1) {
                        const uint32_t amax = mx_quad_max(mx_amax8(v[u][0]));
                        s = mx_scale_byte<kE2M1>(amax);
                        code = mx_encode8_e2m1(v[u][0], amax, s);
                    } else {
                        const float4 x0 = __builtin_bit_cast(float4, v[u][0]);
                        const float4 x1 = __builtin_bit_cast(float4, v[u][SRC - 1]);
                        float f[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                        const uint32_t amax = mx_quad_max(mx_amax8(f));
                        s = mx_scale_byte<kE2M1>(amax);
                        code = mx_encode8_e2m1(f, amax, s);
                    }
                    const int k = ii[u] >> 2, at = (k >> 3) * MR + mi[u];
                    *reinterpret_cast<uint32_t*>(sA + at * 128 + 16 * ((k & 7) ^ ((mi[u] >> 1) & 7)) + 4 * (ii[u] & 3)) = code;
                    if ((ii[u] & 3) == 0) xA[at * 8 + (k & 7)] = (uint8_t)s;
                }
            }
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        for (int t = w; t < nt; t += kFewWaves) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int64_t k = (int64_t)(t0 + t) * 8 + 4 * s + kq;  // this lane's block
                const bool live = k < Ks;
                uint4 fb = *reinterpret_cast<const uint4*>(sB + (t * 16 + row) * 128 + 16 * ((4 * s + kq) ^ (row >> 1)));
                uint4 fa = *reinterpret_cast<const uint4*>(sA + (t * MR + ma) * 128 + 16 * ((4 * s + kq) ^ (ma >> 1)));
                uint32_t xb = *reinterpret_cast<const uint32_t*>(xB + (t * 16 + row) * 8 + 4 * s) >> (8 * kq);
                uint32_t xa = *reinterpret_cast<const uint32_t*>(xA + (t * MR + ma) * 8 + 4 * s) >> (8 * kq);
                if (!live) {  // a block past K
                    fa = make_uint4(0, 0, 0, 0);
                    fb = fa;
                    xa = xb = 127;
                }
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(fb), frag(fa), acc, kFp4, kFp4, 0,
                                                                       (int)xb, 0, (int)xa);
            }
        }
    }
    // D: row (of b) 4 (lane / 16) + v, column (row of a) lane % 16
#pragma unroll
    for (int v = 0; v < 4; ++v) sR[w][row][4 * kq + v] = acc[v];
    __syncthreads();
    // 8 columns per thread: 2 threads per row of a
    if (tid < 32) {
        const int64_t m = m0 + (tid >> 1), nn = n0 + 8 * (tid & 1);
        if (m < p.M && nn < p.N) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float s = 0.f;
#pragma unroll
                for (int ww = 0; ww < kFewWaves; ++ww) s += sR[ww][tid >> 1][8 * (tid & 1) + e];
                y[e] = s;
            }
            if constexpr (EPI == kWriteBack) {
                uint4 xq[4];
                load_x8(p, m, nn / 8, xq);
                write_back8(p, m, nn / 8, y, xq,
                            {map_part(p, m, 0), map_part(p, m, 1), map_part(p, m, 2), map_part(p, m, 3),
                             map_part(p, m, 4)});
            } else {
                store8<EPI>(p, m, nn, y);
            }
        }
    }
}

template <int TM, int TN, int WM, int WN, int NBUF, int EPI>
void tile_as(const Mx4Args& p, hipStream_t stream)
{
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
    const unsigned gm = (unsigned)((p.M + BM - 1) / BM), gn = (unsigned)((p.N + BN - 1) / BN);
    const dim3 block(64 * WM * WN);
    auto* kernel = p.K % (2 * kStageK) == 0 ? mx4_tile_kernel<TM, TN, WM, WN, NBUF, EPI, kPairs>
                   : p.K % kStageK == 0     ? mx4_tile_kernel<TM, TN, WM, WN, NBUF, EPI, kWordwise>
                                          : mx4_tile_kernel<TM, TN, WM, WN, NBUF, EPI, kTail>;
    hipLaunchKernelGGL(kernel, dim3(gm * gn), block, 0, stream, p, gm, gn);
}

// Panels sized for two workgroups per compute unit.
FewShape few_shape(int64_t M, int64_t K)
{
    FewShape s{1, 0, 0, (unsigned)((M + 15) / 16), 0};
    for (; s.MR < 16 && s.MR < M; s.MR *= 2) ++s.LR;
    const int64_t tiles = (K + 255) / 256, most = 70 * 1024 / few_tile_bytes(s.MR);
    const int64_t panels = (tiles + most - 1) / most;
    s.PT = (int)((tiles + panels - 1) / panels);
    s.lds = (unsigned)(s.PT * few_tile_bytes(s.MR));
    return s;
}

template <int SRC, int EPI>
void few_as(const Mx4Args& p, hipStream_t stream)
{
    const FewShape sh = few_shape(p.M, p.K);
    hipLaunchKernelGGL((mx4_few_kernel<SRC, EPI>), dim3((unsigned)((p.N + 127) / 128) * 8 * sh.groups),
                       dim3(kFewThreads), sh.lds, stream, p, sh);
}

template <int EPI>
hipError_t matmul_as(const Mx4Args& p, hipStream_t stream)
{
    if (p.M <= 16 || (p.M + 15) / 16 * ((p.N + 15) / 16) <= 512) {
        // As long as all workgroups of 16 x 16 are on the chip at once (two per
        // compute unit) they beat the tiles below, which then leave most of it
        // idle (us, against tiles of 64): 32 x 4096, K = 4096 5.9 / 7.5;
        // 128 x 1024, K = 8192 7.7 / 10.0; but 64 x 4096 (1024 workgroups)
        // 9.0 / 7.2 and 32 x 7168, K = 7168 (896) 13.2 / 9.5.
        few_as<0, EPI>(p, stream);
    } else {
        // Large tiles move the fewest operand bytes per product and win as
        // soon as they cover most of the chip; below that, more tiles.
        // Measured (us, K = 4096 unless named, tiles of 256 / 128 / 64): 4096 x
        // 4096 42 / 55 / 84; 4096 x 3584 35 / 44 / 66; 1024 x 7168, K = 7168 (112
        // tiles of 256) 47 / 37 / 56; 512 x 7168, K = 7168 (224 tiles of 128) 43 /
        // 21.5 / 33; 512 x 4096 (128) 25 / 12.7 / 11.3; 256 x 4096 (64) 25 / 12 /
        // 7.7.  Three stage buffers instead of two pay while a compute unit has
        // one tile (2048 x 2048: 15.5 / 16.5), cost the second workgroup
        // otherwise (4096 x 4096: 64 / 55).
        const int64_t t256 = ((p.M + 255) / 256) * ((p.N + 255) / 256);
        const int64_t t128 = ((p.M + 127) / 128) * ((p.N + 127) / 128);
        if (t256 >= 192)
            tile_as<2, 4, 4, 2, 2, EPI>(p, stream);
        else if (t128 > 256)
            tile_as<2, 2, 2, 2, 2, EPI>(p, stream);
        else if (t128 > 128)
            tile_as<2, 2, 2, 2, 3, EPI>(p, stream);
        else
            tile_as<1, 1, 2, 2, 3, EPI>(p, stream);
    }
    return hipGetLastError();
}

}  // namespace

bool mx4_fuses_quantize(int64_t M, int64_t K)
{
    // beyond this the second launch is cheaper than every workgroup's own pass
    return M <= 16 && M * K <= 32768;
}

hipError_t launch_mx4_matmul(const Packed& a, const Packed& b, void* out, bool f32, int64_t M,
                             int64_t N, int64_t K, hipStream_t stream)
{
    const Mx4Args p{(const uint8_t*)a.codes, a.scales, (const uint8_t*)b.codes, b.scales, out,
                    nullptr, nullptr, nullptr, nullptr, M, N, K};
    return f32 ? matmul_as<kStoreF32>(p, stream) : matmul_as<kStoreBf16>(p, stream);
}

hipError_t launch_mx4_matmul_fused(const void* a, bool a_f32, const Packed& b, void* out, bool f32,
                                   int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    const Mx4Args p{(const uint8_t*)a, nullptr, (const uint8_t*)b.codes, b.scales, out,
                    nullptr, nullptr, nullptr, nullptr, M, N, K};
    auto* few = a_f32 ? (f32 ? few_as<2, kStoreF32> : few_as<2, kStoreBf16>)
                      : (f32 ? few_as<1, kStoreF32> : few_as<1, kStoreBf16>);
    few(p, stream);
    return hipGetLastError();
}

hipError_t launch_mx4_write_back(const Packed& a, const Packed& b, const void* x,
                                 const float* Hpost, const float* Hres, void* x_out, void* f_out,
                                 int64_t T, int64_t C, int64_t K, hipStream_t stream)
{
    const Mx4Args p{(const uint8_t*)a.codes, a.scales, (const uint8_t*)b.codes, b.scales, f_out,
                    (const uint4*)x, Hpost, Hres, (uint4*)x_out, T, C, K};
    return matmul_as<kWriteBack>(p, stream);
}

}  // namespace mhc
