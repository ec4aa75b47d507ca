// Products of MXFP4 matrices (mxfmt.h, e2m1) on the scaled matrix
// instructions of gfx950:  y[m,n] = sum_k a[m,k] b[n,k].
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 by 64 x 32 elements and
// applies both operands' block scales in the same instruction: lane l holds
// the 32 elements (16 bytes) of row l % 32, block l / 32, and one byte of a
// register as that block's scale.  Products of two e2m1 elements are exact,
// the accumulation is fp32.
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

// 8 consecutive columns (n a multiple of 8) of row m of the product.
template <int EPI>
MHC_DEV void finish8(const Mx4Args& p, int64_t m, int64_t n, const float* y)
{
    if (EPI == kStoreF32) {
        float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + m * p.N + n);
        o[0] = make_float4(y[0], y[1], y[2], y[3]);
        o[1] = make_float4(y[4], y[5], y[6], y[7]);
        return;
    }
    const int64_t N8 = p.N / 8, c = n / 8;
    if (EPI == kStoreBf16) {
        reinterpret_cast<uint4*>(p.out)[m * N8 + c] = mx_pack8(y);
        return;
    }
    if (p.out != nullptr) reinterpret_cast<uint4*>(p.out)[m * N8 + c] = mx_pack8(y);
    uint4 xq[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xq[j] = mhc_load_stream(&p.x[(m * 4 + j) * N8 + c]);
    const float4 hp = reinterpret_cast<const float4*>(p.Hpost)[m];
    const float post[4] = {hp.x, hp.y, hp.z, hp.w};
    float xs[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) mx_unpack8(xq[j], xs[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 h = reinterpret_cast<const float4*>(p.Hres)[4 * m + i];
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float s = post[i] * y[e];
            s = __builtin_fmaf(h.x, xs[0][e], s);
            s = __builtin_fmaf(h.y, xs[1][e], s);
            s = __builtin_fmaf(h.z, xs[2][e], s);
            o[e] = __builtin_fmaf(h.w, xs[3][e], s);
        }
        mhc_store_stream(&p.x_out[(m * 4 + i) * N8 + c], mx_pack8(o));
    }
}

// ---------------------------------------------------------------------------
// Tiled product.  Workgroup: 4 waves as 2 x 2, each 32 TM x 32 TN outputs, K
// in stages of 256 (128 bytes of codes and 8 scales per row).
//
// LDS: a stage's rows of 128 bytes as 8 pieces of 16, piece c of row r at
// place c ^ (r % 8), so that the 8 rows a read phase covers fall on different
// banks.  Scales as two words per row, word h holding blocks h, 2 + h, 4 + h,
// 6 + h: a lane (block half h) then has the scales of its 4 steps in one
// register, and the instruction selects the byte.
//
// Pipeline: two LDS buffers and two register sets of fragments.  While step s
// multiplies, step s + 1's fragments are read.  A stage's last fragments are
// in registers before its last step, so the barrier that hands over the next
// stage stands there: behind it the next stage's first fragments are read and
// the copies of the stage after it start into the freed buffer, which gives
// them a whole stage to land.
//
// TAIL: K is no multiple of 256 (blocks past K are zeroed in A, and scale
// rows, which then start at odd addresses, are read by bytes).
// ---------------------------------------------------------------------------
constexpr int kTK = 256;
constexpr int kRowBytes = kTK / 2;
constexpr int kBlock = 256;

// One copy of 16 bytes per lane from global memory straight to LDS: from a
// wave-uniform base plus a lane offset to a wave-uniform LDS address plus 16
// bytes per lane.  It is written as assembly because the compiler, which
// cannot tell the two buffers apart, would wait for all copies before every
// LDS read.  It has no register result; the wait is the vmcnt(0) before the
// barrier that hands the buffer over.
MHC_DEV void copy_to_lds(const uint8_t* base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(lds), "v"(off), "s"(base) : "memory");
}

struct ScaleRegs {
    uint32_t lo, hi;
};

// the 8 scale bytes of one row's stage; `left` of them exist
template <bool TAIL>
MHC_DEV ScaleRegs load_scales(const uint8_t* p, int64_t left)
{
    ScaleRegs r;
    if (!TAIL) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r.lo = v.x;
        r.hi = v.y;
    } else {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 127u;
        r.lo = v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24;
        r.hi = v[4] | v[5] << 8 | v[6] << 16 | v[7] << 24;
    }
    return r;
}

MHC_DEV void store_scales(uint32_t* lds, int r, const ScaleRegs& s)
{
    // blocks 0 2 4 6 and 1 3 5 7
    *reinterpret_cast<uint2*>(lds + 2 * r) =
        make_uint2(mx_perm(s.hi, s.lo, 0x06040200u), mx_perm(s.hi, s.lo, 0x07050301u));
}

template <int TM, int TN>
struct Frags {
    uint4 a[TM], b[TN];
};

template <int S, bool TAIL, int TM, int TN>
MHC_DEV void read_frags(Frags<TM, TN>& f, const uint8_t* sA, const uint8_t* sB, int ra, int rb,
                        int kh, int64_t left)
{
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = ra + 32 * i;
        f.a[i] = *reinterpret_cast<const uint4*>(sA + r * kRowBytes + 16 * ((2 * S + kh) ^ (r & 7)));
        if (TAIL && left <= 2 * S) f.a[i] = make_uint4(0, 0, 0, 0);  // a block past K
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int r = rb + 32 * j;
        f.b[j] = *reinterpret_cast<const uint4*>(sB + r * kRowBytes + 16 * ((2 * S + kh) ^ (r & 7)));
    }
}

template <int S, int TM, int TN>
MHC_DEV void mma_one(const Frags<TM, TN>& f, const uint32_t (&xa)[TM], const uint32_t (&xb)[TN],
                     f32x16 (&acc)[TM][TN], int i, int j)
{
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        frag(f.a[i]), frag(f.b[j]), acc[i][j], kFp4, kFp4, S, (int)xa[i], S, (int)xb[j]);
}

template <int S, int TM, int TN>
MHC_DEV void mma_step(const Frags<TM, TN>& f, const uint32_t (&xa)[TM], const uint32_t (&xb)[TN],
                      f32x16 (&acc)[TM][TN])
{
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) mma_one<S>(f, xa, xb, acc, i, j);
}

template <int TM, int TN, int EPI, bool TAIL>
__global__ __launch_bounds__(kBlock) void mx4_tile_kernel(Mx4Args p, unsigned gm, unsigned gn)
{
    constexpr int BM = 64 * TM, BN = 64 * TN;
    constexpr int kBytes = (BM + BN) * kRowBytes;  // codes of one stage
    constexpr int kPitch = 32 * TN + 4;            // floats per staged output row
    static_assert(4 * 32 * kPitch * 4 <= 2 * kBytes, "output strips fit the stage buffers");
    __shared__ __attribute__((aligned(16))) uint8_t sC[2][kBytes];
    __shared__ __attribute__((aligned(8))) uint32_t sX[2][2 * (BM + BN)];
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
    const int ra = 32 * TM * (w & 1) + (lane & 31), rb = 32 * TN * (w >> 1) + (lane & 31);
    const int kh = lane >> 5;
    const int stages = (int)((p.K + kTK - 1) / kTK);

    // A thread copies piece c of rows 32 i + tid / 8 (its place in LDS is fixed
    // by tid).  Rows past the matrix repeat its last one; their products are
    // not used.  Row offsets fit 32 bits: 255 rows of at most 2^23 bytes.
    constexpr int NA = 2 * TM, NB = 2 * TN;  // copies per thread and stage
    const int c16 = 16 * ((tid & 7) ^ ((tid >> 3) & 7));
    const uint8_t* baseA = p.a + m0 * Kb;
    const uint8_t* baseB = p.b + n0 * Kb;
    uint32_t offA[NA], offB[NB];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int64_t r = 32 * i + (tid >> 3), last = p.M - 1 - m0;
        offA[i] = (uint32_t)((r < last ? r : last) * Kb) + c16;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t r = 32 * i + (tid >> 3), last = p.N - 1 - n0;
        offB[i] = (uint32_t)((r < last ? r : last) * Kb) + c16;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&sC[0][0];
    const auto copy = [&](int st, int buf, int i) {  // copy i of stage st
        uint32_t cut = 0;
        if (TAIL) {  // bytes past the row repeat its last piece
            const int64_t over = (int64_t)st * kRowBytes + c16 - (Kb - 16);
            cut = over > 0 ? (uint32_t)over : 0u;
        }
        const bool isA = i < NA;
        const uint8_t* base = (isA ? baseA : baseB) + (int64_t)st * kRowBytes;
        copy_to_lds(base, (isA ? offA[isA ? i : 0] : offB[isA ? 0 : i - NA]) - cut,
                    lds0 + buf * kBytes + 16 * (kBlock * i + 64 * w));
    };
    // scale rows of this thread: row tid + 256 i of A's then B's (a workgroup
    // with fewer rows than threads loads some twice)
    constexpr int SR = (BM + BN + kBlock - 1) / kBlock;
    const uint8_t* sp[SR];
    int sr[SR];
#pragma unroll
    for (int i = 0; i < SR; ++i) {
        sr[i] = (tid + kBlock * i) % (BM + BN);
        const bool isA = sr[i] < BM;
        int64_t r = isA ? m0 + sr[i] : n0 + sr[i] - BM;
        const int64_t n = isA ? p.M : p.N;
        r = r < n ? r : n - 1;
        sp[i] = (isA ? p.as : p.bs) + r * Ks;
    }
    ScaleRegs g[SR];
    const auto load_g = [&](int st) {
#pragma unroll
        for (int i = 0; i < SR; ++i) g[i] = load_scales<TAIL>(sp[i] + 8 * (int64_t)st, Ks - 8 * (int64_t)st);
    };
    const auto settle = [&](int buf) {
#pragma unroll
        for (int i = 0; i < SR; ++i) store_scales(sX[buf], sr[i], g[i]);
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    const auto scales = [&](uint32_t (&va)[TM], uint32_t (&vb)[TN], int buf) {
#pragma unroll
        for (int i = 0; i < TM; ++i) va[i] = sX[buf][2 * (ra + 32 * i) + kh];
#pragma unroll
        for (int j = 0; j < TN; ++j) vb[j] = sX[buf][2 * (BM + rb + 32 * j) + kh];
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    Frags<TM, TN> f0, f1;
    uint32_t xa[TM], xb[TN], ya[TM], yb[TN];
    load_g(0);
#pragma unroll
    for (int i = 0; i < NA + NB; ++i) copy(0, 0, i);
    settle(0);
    // Stages past the last one repeat it and nothing uses them: the loop stays
    // one block, which keeps the products between the copies (the compiler
    // sinks them past a branch, and then nothing overlaps).
    const auto clamped = [&](int st) { return st < stages ? st : stages - 1; };
    load_g(clamped(1));
#pragma unroll
    for (int i = 0; i < NA + NB; ++i) copy(clamped(1), 1, i);
    scales(xa, xb, 0);
    read_frags<0, TAIL>(f0, sC[0], sC[0] + BM * kRowBytes, ra, rb, kh, Ks - kh);
    for (int st = 0; st < stages; ++st) {
        const int buf = st & 1;
        const uint8_t* cA = sC[buf];
        const uint8_t* cB = cA + BM * kRowBytes;
        const int64_t left = Ks - 8 * (int64_t)st - kh;  // blocks from this lane's first one on
        read_frags<1, TAIL>(f1, cA, cB, ra, rb, kh, left);
        __builtin_amdgcn_sched_barrier(0);
        mma_step<0>(f0, xa, xb, acc);
        __builtin_amdgcn_sched_barrier(0);
        read_frags<2, TAIL>(f0, cA, cB, ra, rb, kh, left);
        __builtin_amdgcn_sched_barrier(0);
        mma_step<1>(f1, xa, xb, acc);
        __builtin_amdgcn_sched_barrier(0);
        read_frags<3, TAIL>(f1, cA, cB, ra, rb, kh, left);
        __builtin_amdgcn_sched_barrier(0);
        mma_step<2>(f0, xa, xb, acc);
        __builtin_amdgcn_sched_barrier(0);
        settle(buf ^ 1);
        const uint8_t* nA = sC[buf ^ 1];
        scales(ya, yb, buf ^ 1);
        read_frags<0, TAIL>(f0, nA, nA + BM * kRowBytes, ra, rb, kh, left - 8);
        load_g(clamped(st + 2));
        __builtin_amdgcn_sched_barrier(0);
        constexpr int kPer = (NA + NB + TM * TN - 1) / (TM * TN);  // copies behind each product
#pragma unroll
        for (int q = 0; q < TM * TN; ++q) {
            mma_one<3>(f1, xa, xb, acc, q / TN, q % TN);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = kPer * q; i < kPer * (q + 1) && i < NA + NB; ++i) copy(clamped(st + 2), buf, i);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) xa[i] = ya[i];
#pragma unroll
        for (int j = 0; j < TN; ++j) xb[j] = yb[j];
    }
    // every wave is done with the stage buffers before they hold the outputs
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    // D: column lane % 32, rows (v % 4) + 8 (v / 4) + 4 (lane / 32).  A strip of
    // 32 rows goes through the wave's own LDS to 8 columns per lane.
    float* strip = reinterpret_cast<float*>(&sC[0][0]) + w * 32 * kPitch;
    constexpr int kLanes = 4 * TN;                 // lanes per row
    const int64_t mw = m0 + 32 * TM * (w & 1), nw = n0 + 32 * TN * (w >> 1);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        mhc_wave_lds_fence();  // the previous strip's reads come first
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                strip[((v & 3) + 8 * (v >> 2) + 4 * kh) * kPitch + 32 * j + (lane & 31)] = acc[i][j][v];
        mhc_wave_lds_fence();
#pragma unroll
        for (int q = 0; q < 32 * kLanes / 64; ++q) {
            const int r = (64 / kLanes) * q + lane / kLanes, c = 8 * (lane % kLanes);
            const int64_t m = mw + 32 * i + r, n = nw + c;
            if (m < p.M && n < p.N) {
                const float4 y0 = *reinterpret_cast<const float4*>(&strip[r * kPitch + c]);
                const float4 y1 = *reinterpret_cast<const float4*>(&strip[r * kPitch + c + 4]);
                const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
                finish8<EPI>(p, m, n, y);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows of a (up to 16 MT): bound by reading b once.  A workgroup takes 16
// rows of b and all of a; its 8 waves split K, and within a wave the lane
// quarters (l / 16) split it again: each lane reads a run of consecutive
// blocks of its row.  A sum may take the blocks in any order, so both operands
// only have to agree, and the 16 x 16 x 128 instruction multiplies 4 blocks
// that are not neighbours.  All of a wave's loads of b are issued at once.
// The waves' partial sums meet in LDS and are added in wave order.
//
// SRC 0: a is packed.  SRC 1, 2 (MT = 1): a is bf16 or fp32 and every
// workgroup quantises it for itself into LDS, while its loads of b are in
// flight: one launch instead of two, for a call that lasts a few microseconds.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;
constexpr int kFewRun = 8;  // blocks per lane and pass

template <int MT, int SRC, int EPI>
__global__ __launch_bounds__(64 * kFewWaves) void mx4_few_kernel(Mx4Args p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t sQ[];  // SRC > 0: codes, then scales
    __shared__ float sR[kFewWaves][MT][16][17];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int row = lane & 15, kq = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t Ks = p.K / 32, Kb = p.K / 2;
    const int64_t per = (Ks + 4 * kFewWaves - 1) / (4 * kFewWaves);
    const int64_t first = (4 * w + kq) * per;  // this lane's run of blocks
    int64_t n = n0 + row;
    n = n < p.N ? n : p.N - 1;
    const uint8_t* bc = p.b + n * Kb;
    const uint8_t* bx = p.bs + n * Ks;
    uint4 fb[kFewRun];
    uint32_t xb[kFewRun];
    const auto load_b = [&](int64_t at) {
#pragma unroll
        for (int s = 0; s < kFewRun; ++s) {
            int64_t k = first + at + s;
            k = k < Ks ? k : Ks - 1;
            const mhc_u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const mhc_u32x4*>(bc + 16 * k));
            fb[s] = make_uint4(v.x, v.y, v.z, v.w);
            xb[s] = bx[k];
        }
    };
    uint8_t* qx = sQ + p.M * Kb;
    if (SRC == 0) {
        load_b(0);
    } else {
        // quantise a: 8 columns per lane, a block per quad.  The first pieces
        // are loaded before b, since loads complete in order.
        constexpr int kPre = 2, kThreads = 64 * kFewWaves;
        const int64_t chunks = p.M * (p.K / 8);
        const uint4* av = reinterpret_cast<const uint4*>(p.a);
        const auto quantise = [&](int64_t c, uint4 q, uint4 q2) {
            uint32_t code, s;
            if (SRC == 1) {
                const uint32_t amax = mx_quad_max(mx_amax8(q));
                s = mx_scale_byte<kE2M1>(amax);
                code = mx_encode8_e2m1(q, amax, s);
            } else {
                const float4 u = __builtin_bit_cast(float4, q), v = __builtin_bit_cast(float4, q2);
                float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
                const uint32_t amax = mx_quad_max(mx_amax8(f));
                s = mx_scale_byte<kE2M1>(amax);
                code = mx_encode8_e2m1(f, amax, s);
            }
            reinterpret_cast<uint32_t*>(sQ)[c] = code;
            if ((c & 3) == 0) qx[c >> 2] = (uint8_t)s;
        };
        uint4 pre[kPre][SRC > 0 ? SRC : 1];
#pragma unroll
        for (int i = 0; i < kPre; ++i) {
            int64_t c = tid + kThreads * i;
            c = c < chunks ? c : chunks - 1;
#pragma unroll
            for (int h = 0; h < SRC; ++h) pre[i][h] = av[SRC * c + h];
        }
        __builtin_amdgcn_sched_barrier(0);
        load_b(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kPre; ++i)
            if (tid + kThreads * i < chunks) quantise(tid + kThreads * i, pre[i][0], pre[i][SRC - 1]);
        for (int64_t c = tid + kThreads * kPre; c < chunks; c += kThreads)
            quantise(c, av[SRC * c], av[SRC * c + SRC - 1]);
        mhc_lds_barrier();
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t at = 0;;) {
#pragma unroll
        for (int s = 0; s < kFewRun; ++s) {
            const int64_t k = first + at + s;
            const bool live = at + s < per && k < Ks;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t m = 16 * t + row;
                uint4 fa = make_uint4(0, 0, 0, 0);
                uint32_t xa = 127;
                if (live && m < p.M) {
                    if (SRC > 0) {
                        fa = *reinterpret_cast<const uint4*>(sQ + m * Kb + 16 * k);
                        xa = qx[m * Ks + k];
                    } else {
                        fa = *reinterpret_cast<const uint4*>(p.a + m * Kb + 16 * k);
                        xa = p.as[m * Ks + k];
                    }
                }
                // a dead block is zero in a, and its (repeated) scale of b is
                // replaced, so that a NaN there stays out
                acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    frag(fb[s]), frag(fa), acc[t], kFp4, kFp4, 0, live ? (int)xb[s] : 127, 0, (int)xa);
            }
        }
        at += kFewRun;
        if (at >= per) break;
        load_b(at);
    }
    // D: row (of b) 4 (lane / 16) + v, column (row of a) lane % 16
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) sR[w][t][row][4 * kq + v] = acc[t][v];
    __syncthreads();
    // 8 columns per thread: 2 threads per row of a
    if (tid < 32 * MT) {
        const int64_t m = tid >> 1, nn = n0 + 8 * (tid & 1);
        if (m < p.M && nn < p.N) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float s = 0.f;
#pragma unroll
                for (int ww = 0; ww < kFewWaves; ++ww) s += sR[ww][tid >> 5][(tid >> 1) & 15][8 * (tid & 1) + e];
                y[e] = s;
            }
            finish8<EPI>(p, m, nn, y);
        }
    }
}

template <int TM, int TN, int EPI>
void tile_as(const Mx4Args& p, hipStream_t stream)
{
    const unsigned gm = (unsigned)((p.M + 64 * TM - 1) / (64 * TM));
    const unsigned gn = (unsigned)((p.N + 64 * TN - 1) / (64 * TN));
    if (p.K % kTK == 0)
        hipLaunchKernelGGL((mx4_tile_kernel<TM, TN, EPI, false>), dim3(gm * gn), dim3(kBlock), 0,
                           stream, p, gm, gn);
    else
        hipLaunchKernelGGL((mx4_tile_kernel<TM, TN, EPI, true>), dim3(gm * gn), dim3(kBlock), 0,
                           stream, p, gm, gn);
}

template <int MT, int SRC, int EPI>
void few_as(const Mx4Args& p, hipStream_t stream)
{
    const unsigned lds = SRC > 0 ? (unsigned)(p.M * (p.K / 2 + p.K / 32)) : 0u;
    hipLaunchKernelGGL((mx4_few_kernel<MT, SRC, EPI>), dim3((unsigned)((p.N + 15) / 16)),
                       dim3(64 * kFewWaves), lds, stream, p);
}

template <int EPI>
hipError_t matmul_as(const Mx4Args& p, int src, hipStream_t stream)
{
    if (src == 1) {
        few_as<1, 1, EPI>(p, stream);
    } else if (src == 2) {
        few_as<1, 2, EPI>(p, stream);
    } else if (p.M <= 16) {
        few_as<1, 0, EPI>(p, stream);
    } else if (p.M <= 32) {
        few_as<2, 0, EPI>(p, stream);
    } else if (p.M <= 64) {
        few_as<4, 0, EPI>(p, stream);
    } else {
        // the largest tile that still gives every compute unit one
        const int64_t t256 = ((p.M + 255) / 256) * ((p.N + 255) / 256);
        const int64_t t128 = ((p.M + 127) / 128) * ((p.N + 127) / 128);
        if (t256 >= 256)
            tile_as<4, 4, EPI>(p, stream);
        else if (t128 >= 256)
            tile_as<2, 2, EPI>(p, stream);
        else
            tile_as<1, 1, EPI>(p, stream);
    }
    return hipGetLastError();
}

}  // namespace

bool mx4_fuses_quantize(int64_t M, int64_t K)
{
    return M <= 16 && M * (K / 2 + K / 32) <= 48 * 1024;
}

hipError_t launch_mx4_matmul(const Packed& a, const Packed& b, void* out, bool f32, int64_t M,
                             int64_t N, int64_t K, hipStream_t stream)
{
    const Mx4Args p{(const uint8_t*)a.codes, a.scales, (const uint8_t*)b.codes, b.scales, out,
                    nullptr, nullptr, nullptr, nullptr, M, N, K};
    return f32 ? matmul_as<kStoreF32>(p, 0, stream) : matmul_as<kStoreBf16>(p, 0, stream);
}

hipError_t launch_mx4_matmul_fused(const void* a, bool a_f32, const Packed& b, void* out, bool f32,
                                   int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    const Mx4Args p{(const uint8_t*)a, nullptr, (const uint8_t*)b.codes, b.scales, out,
                    nullptr, nullptr, nullptr, nullptr, M, N, K};
    const int src = a_f32 ? 2 : 1;
    return f32 ? matmul_as<kStoreF32>(p, src, stream) : matmul_as<kStoreBf16>(p, src, stream);
}

hipError_t launch_mx4_write_back(const Packed& a, const Packed& b, const void* x,
                                 const float* Hpost, const float* Hres, void* x_out, void* f_out,
                                 int64_t T, int64_t C, int64_t K, hipStream_t stream)
{
    const Mx4Args p{(const uint8_t*)a.codes, a.scales, (const uint8_t*)b.codes, b.scales, f_out,
                    (const uint4*)x, Hpost, Hres, (uint4*)x_out, T, C, K};
    return matmul_as<kWriteBack>(p, 0, stream);
}

}  // namespace mhc
