// decode_attn_paged over a pool of 4 bits (q4_0).
//
// Every code is read once and used for the G query heads of its group: 72 bytes for 128 values, and so little of them that
// what bounds it is turning nibbles into operands.  Two things keep that short.
//   - An fp16 number is linear in its bits as long as the exponent's are zero, and matrix products take such numbers exactly:
//     a nibble n (code + 8) in the low byte of a half is the subnormal n 2^-24 or n 2^-20 where it lies.  An AND with
//     0x000F000F or 0x00F000F0 makes two operands, and no subtraction or conversion is left to do for each value.  In the first
//     product the queries of the lower nibbles are 16 times as large, in the second the sums of the upper ones are.
//   - The 8 in each nibble is taken care of outside of the loops over values: the scores begin at -8 times the product of
//     the key's scales with the sums of the queries over each block (one small product, the sums in two fp16 parts), and a
//     product with eights in place of the values is subtracted from O after every FOLD tiles.  Left in O, the eights would be most
//     of it, and float32 sums of matrix products, which cut toward zero, count against all of it: with whole bytes n + 16 n' summed to
//     the end of a run of 16,384 keys, V's scales of one sign, float32 outputs were off by 2.1e-3 of their rms (65,536 keys
//     4.4e-3; scales of either sign 3.4e-4 and 6.5e-4).  They are off by 1.7e-5 and 6.6e-5, and by 2.0e-4 and 2.1e-4, which is
//     fp16 numerators'.  It takes 1.2 us of the 96 sequences below in bf16 (FOLD 1, 4 and 8: 55.3, 54.2 and 54.0 us; signed codes as
//     operands, 1024 + n less 1032: 57.9), 4 of the 82 in 16 heads to a group.
// V's scales are multiplied into the numerators: in float32, before their one rounding, or where the output is bf16, whose
// rounding is eight times as coarse, in fp16, after one.  All of these stay in fp16's range: a head's numerators are 2^7 to
// 2^11 at its greatest score, and a warp takes the scales of each block times a power of two (factor) that brings the greatest that
// it has met to 2^3 or more, below 2^4 (or any to 2^15 times itself).  So numerators count down to 2^-31 of the greatest, and scales to
// 2^-28, with all of their bits to 2^-17.  (Scales of at most one beside numerators of up to 2^15 lost bits from 2^-14 on and
// vanished at 2^-25, whatever their keys weighed.  Numerators of up to 2^8 beside scales of up to 2^7: one of eight heads passes its
// limit so often that the 96 sequences below take 2 us more; products in float32 for bf16 outputs too: the same.)
//
// Work split.  The list of decode_attn_paged, in tiles of 32 keys, is cut into runs for single *warps*: a warp looks up its
// pages, keeps its own ring of tiles in flight and attends over them with all heads of the group and all dimensions; warps
// share nothing but the look at the lengths, and starting and ending a pair holds up one warp.  (With four warps
// on a pair's tiles and a fifth that loads, as for f16 and q8_0 pools, a pair's start and end took 2 us, which the four times
// shorter tiles did not hide: the 96 sequences below 67 us.)  The four warps of a CTA (two, one where the kv heads
// do not divide) take the same tokens of neighbouring kv heads, whose codes lie side by side in a layer-major pool: 58 us
// instead of 67.  Copies are 16-byte asynchronous ones, waited for by the warp itself; no wait can fail to end.
// TMA took 5 cycles for each row of 64 bytes, and 47 us where nothing was computed.
//
// Measured (40 query heads, 8 kv heads of 128, bf16, calls back to back in a graph; of the rate of a copy): 96 sequences of 5
// to 16,384 tokens 54.3 us (3.8 TB/s, 0.56; to fp16 56.3, float32 56.9; the same from q8_0 82), in 16 heads to a group 87.4; 20 of
// 16,384 78 (0.71), 96 of them 345 (0.77); one of 58,300 22.7 us (0.44); eight of about 2,100 14.0; one of 64 8.0.  Where the 96 took
// 53, before the eights were folded, the warps' runs took 43 on average and 47.5 at most, the join and the launches 6; without
// the products all of it took 45.  A tile took a scheduler about 1,100 cycles, in which it issued 570 instructions: 42 matrix
// instructions, each 8 cycles of the tensor pipe and about four in which nothing else issues, and 390 others for the products,
// 140 to ask for the next tile; three warps do not hide the rest of the chain product - maximum - exponential - product.
#include "decode_paged.cuh"

namespace kvc {
namespace {

using namespace paged;

constexpr int KT = 32;              // keys per tile: two subtiles of 16, each within one page
constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
// What starting and ending a pair costs, in tiles.  With 1, 2, 3, 4 and 6, in us: the 96 sequences 62.4, 57.4, 53.7, 53.9 and 55.2,
// 170 of up to 3,000 21.4, 21.1, 20.3, 20.0 and 20.5.
constexpr int PIECE_COST = 4;
// CTAs per SM: as many as the registers allow (three 168, of which those for heads of 128 and 16-bit queries take all; nothing
// spills).  Two instead of three: the 96 sequences 57.5 us, in heads of 64 48 instead of 39; four (128 registers) 64.
constexpr int ctas_per_sm(int NT) { return NT == 1 ? 3 : 2; }
constexpr int MAX_NS = 6;
constexpr int FOLD = 4;             // tiles between two subtractions of the eights from O: a power of two
constexpr float NONE = -1e30f;      // the reference of a head that has met no key
constexpr float RAISE_LOG2 = SHIFT_LOG2 + 4.0f;   // a numerator above 2^this raises its head's reference

// A warp's way through its run of the list: groups of kv heads, in each the sequences, in each its units.  Kept in shared
// memory, where the loop over tiles leaves it alone: registers decide how many warps there are.
struct Way {
    unsigned long long left;
    int seq, group, x, base;     // x: units of the current pair that lie before this run
    int held[32];                // lengths from sequence `base` on
    Piece piece;                 // h: the group
};

// A CTA's shared memory besides its warps' tiles.
struct Small {
    unsigned long long warp_units[WARPS], units_before[THREADS];
    Way ways[WARPS][2];
    int lengths[THREADS];        // of all sequences, where they are so few
};
constexpr int SMALL = (sizeof(Small) + 127) / 128 * 128;

template <int D, int DT, int NT>
struct Cfg {
    static constexpr bool FINE = DT != KVC_IN_BF16;
    static constexpr int U = NT == 1 ? 2 : 1;               // subtiles taken together
    static constexpr uint32_t ALL = U == 2 ? 0xFFFFFFFFu : 0xFFFFu;
    static constexpr int NB = D / 32;                       // blocks per row
    static constexpr int ROW = D / 2;                       // bytes of a row
    static constexpr int TILE = KT * ROW;                   // a K or V tile
    static constexpr int SC = KT * NB * 2;                  // a tile's scales
    static constexpr int STAGE = 2 * TILE + 2 * SC;         // keeps the tiles on the swizzle's boundaries
    static constexpr int MT = D / 16;                       // 16-row tiles of O^T
    // of 228 KB, 1 KB for each CTA besides what it asks for; for heads of 128 three CTAs leave nothing over
    static constexpr int FIT = (228 * 1024 / ctas_per_sm(NT) - 1024 - SMALL) / (WARPS * STAGE);
    static constexpr int NS = FIT < MAX_NS ? FIT : MAX_NS;
    static constexpr int SMEM = WARPS * NS * STAGE;
    static_assert(ctas_per_sm(NT) * (SMEM + SMALL + 1024) <= 228 * 1024, "the CTAs that slots are counted by have to fit an SM");
    static constexpr int CHUNKS = ROW / 16, RPL = 32 / CHUNKS;   // 16-byte chunks of a row; rows that a warp's copy takes
    static_assert(NS >= 2, "shared memory plan");
};

// Which chunk of a row lies in place c: eight rows' chunks c lie in all banks.
template <int D>
__device__ __forceinline__ int swizzle(int row, int c) { return D == 128 ? c ^ ((row >> 1) & 3) : c ^ ((row >> 2) & 1); }

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, int bytes) {   // 16, or 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_scales(uint32_t dst, const uint8_t *src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(valid ? N : 0) : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups_but() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The power of two that brings |d| to 2^3 or more, below 2^4; 2^15 at most.
__device__ __forceinline__ __half factor_of(__half d) {
    const int e = min(__half_as_ushort(d) >> 10 & 31, 30);   // |d| < 2^(e - 14)
    return __ushort_as_half((unsigned short)(min(33 - e, 30) << 10));
}

// A lane's values of the group's queries, eight of each block, as they lie in memory.
template <int D, int DT, int NT>
struct RawQueries {
    uint4 u[NT][D / 32][DT == KVC_IN_F32 ? 2 : 1];
};
template <int D, int DT, int NT>
__device__ __forceinline__ void read_queries(const uint8_t *q, int G, int lane, RawQueries<D, DT, NT> &raw) {
    constexpr int ESZ = DT == KVC_IN_F32 ? 4 : 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int head = nt * 8 + (lane >> 2);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            const uint4 *at = reinterpret_cast<const uint4 *>(q + (head * D + 32 * b + 8 * (lane & 3)) * ESZ);
#pragma unroll
            for (int i = 0; i < (DT == KVC_IN_F32 ? 2 : 1); ++i) raw.u[nt][b][i] = head < G ? __ldcg(at + i) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
}
template <int DT>
__device__ __forceinline__ void widen_q(const uint4 *u, float (&v)[8]) {
    const uint4 x = u[0];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (DT == KVC_IN_F32) {
        const uint4 y = u[1];
        const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = __uint_as_float(w[i]); v[4 + i] = __uint_as_float(z[i]); }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = DT == KVC_IN_F16 ? __half22float2(as_half2(w[i]))
                                              : make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// The group's queries, each head scaled by a power of two (its greatest magnitude to 2^14, 2^10 for upper nibbles): any
// magnitude from 2^-100 to 2^100 keeps its 11 bits.  eights: the second operand of the product that the scores begin
// with, worth: what this lane's two columns' products are worth in powers of two.
template <int D, int DT, int NT>
__device__ __forceinline__ void make_queries(const RawQueries<D, DT, NT> &raw, float scale_log2, int lane,
                                             uint32_t (&qf)[D / 16][NT][2], uint32_t (&eights)[NT], float (&worth)[NT][2]) {
    const int t4 = lane & 3;
    constexpr int NB = D / 32;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float v[NB][8], most = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) widen_q<DT>(raw.u[nt][b], v[b]);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 8; i += 2) most = fmax3(most, fabsf(v[b][i]), fabsf(v[b][i + 1]));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const int ex = most > 0.f ? min(max((int)(__float_as_uint(most) >> 23) - 127, -100), 100) : 0;
        const float lo = __uint_as_float((uint32_t)(127 + 10 - ex) << 23), hi = 16.f * lo;
        const float w = __uint_as_float((uint32_t)(127 + 10 + ex) << 23) * scale_log2;
#pragma unroll
        for (int e = 0; e < 2; ++e) worth[nt][e] = __shfl_sync(0xffffffffu, w, (2 * t4 + e) * 4);
        float sum[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            sum[b] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t p = pack_half2(v[b][2 * i] * (i & 1 ? lo : hi), v[b][2 * i + 1] * (i & 1 ? lo : hi));
                const float2 f = __half22float2(as_half2(p));
                sum[b] += (f.x + f.y) * (i & 1 ? 1.f : 0.0625f);
                qf[2 * b + (i >> 1)][nt][i & 1] = p;
            }
        }
#pragma unroll
        for (int x = 1; x < 4; x <<= 1)
#pragma unroll
            for (int b = 0; b < NB; ++b) sum[b] += __shfl_xor_sync(0xffffffffu, sum[b], x);
        float mine[2] = {sum[0], sum[1]};   // of blocks 2 t4 and 2 t4 + 1, and again from lane NB / 2 on
        if (NB == 4 && (t4 & 1)) { mine[0] = sum[NB - 2]; mine[1] = sum[NB - 1]; }
        mine[0] *= -0x1p-17f;               // eight of the upper nibbles' units
        mine[1] *= -0x1p-17f;
        const uint32_t p = pack_half2(mine[0], mine[1]);
        const float2 f = __half22float2(as_half2(p));
        const uint32_t rest = pack_half2(mine[0] - f.x, mine[1] - f.y);
        eights[nt] = t4 < NB / 2 ? p : t4 < NB ? rest : 0u;
    }
}

// U subtiles of a tile, from row `row0` on: scores, numerators, sums.  exists: a bit for each of their keys.
template <int D, int NT, class C>
__device__ __forceinline__ void attend(uint32_t kt, int row0, uint32_t exists, int lane, const uint32_t (&qf)[D / 16][NT][2],
                                       const uint32_t (&eights)[NT], const float (&worth)[NT][2], float (&o)[C::MT][NT][4],
                                       float (&ob)[C::NB][NT][4], float (&m)[NT][2], float (&l)[NT][2],
                                       __half2 (&factor)[C::NB / 2]) {
    constexpr int U = C::U, NB = C::NB;
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t vt = kt + C::TILE, sc = vt + C::TILE;
    const int g = lane >> 2, t4 = lane & 3;
    // ldmatrix: lane i names row i % 8 of matrix i / 8: keys 0 to 7 and 8 to 15 of a block (16 bytes), then of the next one
    const int mrow = (lane & 7) + 8 * ((lane >> 3) & 1), mchunk = lane >> 4;
    uint32_t kw[U][NB / 2][4], vw[U][NB / 2][4];
    __half2 dk[U][2][NB / 2], dv[U][2][NB / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
            const int sw = swizzle<D>(mrow, b + mchunk);
            ldmatrix_x4(kw[u][b >> 1], kt + (row0 + u * 16 + mrow) * C::ROW + (sw << 4));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = sc + (row0 + u * 16 + g + 8 * h) * (2 * NB);
            if constexpr (NB == 4) {
                const uint2 x = lds64(at), y = lds64(at + C::SC);
                dk[u][h][0] = as_half2(x.x); dk[u][h][1] = as_half2(x.y);
                dv[u][h][0] = as_half2(y.x); dv[u][h][1] = as_half2(y.y);
            } else {
                dk[u][h][0] = as_half2(lds32(at));
                dv[u][h][0] = as_half2(lds32(at + C::SC));
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
            const int sw = swizzle<D>(mrow, b + mchunk);
            ldmatrix_x4_trans(vw[u][b >> 1], vt + (row0 + u * 16 + mrow) * C::ROW + (sw << 4));
        }
    float s[U][NT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        // the scales of blocks 2 t4 and 2 t4 + 1, and again from lane NB / 2 on, as the sums of the queries lie
        const uint32_t da = as_u32(NB == 4 && (t4 & 1) ? dk[u][0][NB / 2 - 1] : dk[u][0][0]);
        const uint32_t db = as_u32(NB == 4 && (t4 & 1) ? dk[u][1][NB / 2 - 1] : dk[u][1][0]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_1688_to(s[u][nt], da, db, eights[nt], zero);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t ka = kw[u][b >> 1][2 * (b & 1)], kb = kw[u][b >> 1][2 * (b & 1) + 1], ka8 = ka >> 8, kb8 = kb >> 8;
            const uint32_t A[4] = {ka & LO, kb & LO, ka & HI, kb & HI}, B[4] = {ka8 & LO, kb8 & LO, ka8 & HI, kb8 & HI};
            const float ca = __half2float(b & 1 ? __high2half(dk[u][0][b >> 1]) : __low2half(dk[u][0][b >> 1]));
            const float cb = __half2float(b & 1 ? __high2half(dk[u][1][b >> 1]) : __low2half(dk[u][1][b >> 1]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float acc[4];
                mma_16816_to(acc, A, qf[2 * b][nt][0], qf[2 * b][nt][1], zero);
                mma_16816_to(acc, B, qf[2 * b + 1][nt][0], qf[2 * b + 1][nt][1], acc);
                f2_unpack(f2_fma(f2_pack(acc[0], acc[1]), f2_pack(ca, ca), f2_pack(s[u][nt][0], s[u][nt][1])), s[u][nt][0], s[u][nt][1]);
                f2_unpack(f2_fma(f2_pack(acc[2], acc[3]), f2_pack(cb, cb), f2_pack(s[u][nt][2], s[u][nt][3])), s[u][nt][2], s[u][nt][3]);
            }
        }
        // In powers of two, and rounded before the reference is taken off, as the reference was: fused, the greatest score less its
        // reference would be off by the reference's rounding, which passes any exponent where scores pass 2^27.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint64_t w2 = f2_pack(worth[nt][0], worth[nt][1]);
            f2_unpack(f2_mul(f2_pack(s[u][nt][0], s[u][nt][1]), w2), s[u][nt][0], s[u][nt][1]);
            f2_unpack(f2_mul(f2_pack(s[u][nt][2], s[u][nt][3]), w2), s[u][nt][2], s[u][nt][3]);
        }
    }
    if (exists != C::ALL) {   // the last subtile of a sequence, or one of a hole
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (!(exists >> (16 * u + g) & 1)) s[u][nt][0] = s[u][nt][1] = -INFINITY;
                if (!(exists >> (16 * u + g + 8) & 1)) s[u][nt][2] = s[u][nt][3] = -INFINITY;
            }
    }
    bool above = false;
    __half2 d_here[NB / 2];   // the greatest scales of V; is one too large for its block's factor?
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) {
        d_here[i] = __hmax2(__habs2(dv[0][0][i]), __habs2(dv[0][1][i]));
#pragma unroll
        for (int u = 1; u < U; ++u) d_here[i] = __hmax2(d_here[i], __hmax2(__habs2(dv[u][0][i]), __habs2(dv[u][1][i])));
        above |= !__hble2(__hmul2(d_here[i], factor[i]), __float2half2_rn(16.f));
    }
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[nt][e] = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
#pragma unroll
            for (int u = 1; u < U; ++u) top[nt][e] = fmax3(top[nt][e], s[u][nt][e], s[u][nt][e + 2]);
            above |= top[nt][e] - m[nt][e] > RAISE_LOG2;
        }
    if (__any_sync(0xffffffffu, above)) {
        float fb[NB];
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
                d_here[i] = __hmax2(d_here[i], as_half2(__shfl_xor_sync(0xffffffffu, as_u32(d_here[i]), x)));
            const float2 was = __half22float2(factor[i]);
            factor[i] = __hmin2(factor[i], __halves2half2(factor_of(__low2half(d_here[i])), factor_of(__high2half(d_here[i]))));
            const float2 is = __half22float2(factor[i]);
            fb[2 * i] = is.x / was.x;
            fb[2 * i + 1] = is.y / was.y;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = top[nt][e];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                // only heads that are above it: what a head's numerators are does not depend on other heads
                const float m_new = x - m[nt][e] > RAISE_LOG2 ? x - SHIFT_LOG2 : m[nt][e];
                f[e] = ex2(m[nt][e] - m_new);
                m[nt][e] = m_new;
                l[nt][e] *= f[e];
            }
#pragma unroll
            for (int i = 0; i < C::MT; ++i) {
                const float f0 = f[0] * fb[i >> 1], f1 = f[1] * fb[i >> 1];
                o[i][nt][0] *= f0; o[i][nt][1] *= f1; o[i][nt][2] *= f0; o[i][nt][3] *= f1;
                if (i & 1) { ob[i >> 1][nt][0] *= f0; ob[i >> 1][nt][1] *= f1; }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t pe[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                float x0, x1;
                f2_unpack(f2_add(f2_pack(s[u][nt][i], s[u][nt][i + 1]), f2_pack(-m[nt][0], -m[nt][1])), x0, x1);
                s[u][nt][i] = ex2(x0);
                s[u][nt][i + 1] = ex2(x1);
            }
            l[nt][0] += s[u][nt][0] + s[u][nt][2];
            l[nt][1] += s[u][nt][1] + s[u][nt][3];
            if constexpr (!C::FINE) {
                pe[nt][0] = pack_half2(s[u][nt][0], s[u][nt][1]);
                pe[nt][1] = pack_half2(s[u][nt][2], s[u][nt][3]);
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t va = vw[u][b >> 1][2 * (b & 1)], vb = vw[u][b >> 1][2 * (b & 1) + 1], va8 = va >> 8, vb8 = vb >> 8;
            const uint32_t A[4] = {va & LO, va & HI, vb & LO, vb & HI}, B[4] = {va8 & LO, va8 & HI, vb8 & LO, vb8 & HI};
            const uint32_t E[4] = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};
            const __half2 da = __hmul2(dv[u][0][b >> 1], factor[b >> 1]), db = __hmul2(dv[u][1][b >> 1], factor[b >> 1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t p0, p1;
                if constexpr (C::FINE) {
                    const float ca = __half2float(b & 1 ? __high2half(da) : __low2half(da));
                    const float cb = __half2float(b & 1 ? __high2half(db) : __low2half(db));
                    p0 = pack_half2(s[u][nt][0] * ca, s[u][nt][1] * ca);
                    p1 = pack_half2(s[u][nt][2] * cb, s[u][nt][3] * cb);
                } else {
                    p0 = as_u32(__hmul2(as_half2(pe[nt][0]), b & 1 ? __high2half2(da) : __low2half2(da)));
                    p1 = as_u32(__hmul2(as_half2(pe[nt][1]), b & 1 ? __high2half2(db) : __low2half2(db)));
                }
                p0 = movmatrix_trans(p0);
                p1 = movmatrix_trans(p1);
                mma_16816_to(o[2 * b][nt], A, p0, p1, o[2 * b][nt]);
                mma_16816_to(o[2 * b + 1][nt], B, p0, p1, o[2 * b + 1][nt]);
                mma_16816_to(ob[b][nt], E, p0, p1, ob[b][nt]);
            }
        }
    }
}

// The eights leave O: low nibbles' sums (rows 0 to 7 of a tile) have them once, upper ones' 16 times.
template <int NT, class C>
__device__ __forceinline__ void fold_eights(float (&o)[C::MT][NT][4], float (&ob)[C::NB][NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < C::NB; ++b) {
#pragma unroll
            for (int i = 2 * b; i < 2 * b + 2; ++i) {
                o[i][nt][0] -= ob[b][nt][0];
                o[i][nt][1] -= ob[b][nt][1];
                o[i][nt][2] = fmaf(ob[b][nt][0], -16.f, o[i][nt][2]);
                o[i][nt][3] = fmaf(ob[b][nt][1], -16.f, o[i][nt][3]);
            }
            ob[b][nt][0] = ob[b][nt][1] = ob[b][nt][2] = ob[b][nt][3] = 0.f;
        }
}

// Where the layer's codes and scales lie; distances in bytes.
struct Codes {
    const uint8_t *k, *sk;
    int64_t v_from_k, sv_from_sk, head, s_head;
    uint32_t tok, rows, s_tok;   // rows: of the rows that a warp copies together
};

// keys_of, from the CTA's copy of the lengths where it has them all.
__device__ __forceinline__ int keys_at(const PagedView &pg, const int *all, int i) {
    return pg.n_seq <= THREADS ? all[i] : keys_of(pg, i);
}
__device__ __forceinline__ void look(Way *w, const PagedView &pg, const int *all, int seq, int lane) {
    __syncwarp();
    w->held[lane] = seq + lane < pg.n_seq ? keys_at(pg, all, seq + lane) : 0;
    if (lane == 0) w->base = seq;
    __syncwarp();
}
__device__ __forceinline__ void start(Way *w, const PagedView &pg, const int *all, int seq, int group, int x, unsigned long long left,
                                      int lane) {
    if (lane == 0) {
        w->left = left;
        w->seq = seq;
        w->group = group;
        w->x = x;
    }
    look(w, pg, all, seq, lane);
}
// In 32 bits where that is enough: 64-bit divisions take some hundred cycles each.
__device__ __forceinline__ unsigned long long div64(unsigned long long a, unsigned long long b) {
    return (a | b) >> 32 ? a / b : (unsigned)a / (unsigned)b;
}
// The next piece into w->piece; false: there is none.
__device__ __noinline__ bool next(Way *w, const PagedView &pg, const int *lengths, int groups, int lane) {
    unsigned long long left = w->left;
    int seq = w->seq, group = w->group, x = w->x, base = w->base;
    Piece p = {0, 0, 0, 0, 0, 0};
    bool found = false;
    while (!found && left > 0 && group < groups) {
        if (seq - base >= 32 || seq < base) {
            look(w, pg, lengths, seq, lane);
            base = seq;
        }
        const int keys = w->held[seq - base], all = units_of<KT, PIECE_COST>(keys);
        const int x1 = (int)min((unsigned long long)all, x + left);
        p = {seq, group, max(x - PIECE_COST, 0), max(x1 - PIECE_COST, 0), tiles_of<KT>(keys), keys};
        left -= x1 - x;
        x = 0;
        if (++seq == pg.n_seq) { seq = 0; ++group; }
        found = p.t1 > p.t0;
    }
    __syncwarp();
    if (lane == 0) {
        w->left = left;
        w->seq = seq;
        w->group = group;
        w->x = x;
        w->piece = p;
    }
    __syncwarp();
    return found;
}

template <int DT>
__device__ __forceinline__ void store_out8(void *out, int64_t i, const float (&x)[8]) {
    if constexpr (DT == KVC_IN_F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(out) + i);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (DT == KVC_IN_F16) {
                w[j] = pack_half2(x[2 * j], x[2 * j + 1]);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int D, int DT, int NT>
__global__ void __launch_bounds__(THREADS, ctas_per_sm(NT))
    decode_paged_q4_kernel(const PagedView pg, const Args a, const Codes codes) {
    using C = Cfg<D, DT, NT>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ Small small;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    // ---- where the warp's run of the list starts: a.step warps take the heads of a group in one run
    const int groups = a.H_kv / a.step;
    const int c = blockIdx.x * WARPS + warp, member = warp % a.step;   // my slot, my head of a group
    const unsigned run = c / a.step;
    Way *ahead = &small.ways[warp][0], *way = &small.ways[warp][1];
    // each thread takes `per` sequences: the units before its own, in its warp
    const int per = (pg.n_seq + THREADS - 1) / THREADS;
    {
        const int i0 = min((int)threadIdx.x * per, pg.n_seq), i1 = min(i0 + per, pg.n_seq);
        unsigned long long mine = 0;
        for (int i = i0; i < i1; ++i) {
            const int keys = keys_of(pg, i);
            mine += units_of<KT, PIECE_COST>(keys);
            if (per == 1) small.lengths[i] = keys;
        }
        unsigned long long sum = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const unsigned long long up = __shfl_up_sync(0xffffffffu, sum, x);
            if (lane >= x) sum += up;
        }
        if (lane == 31) small.warp_units[warp] = sum;
        small.units_before[threadIdx.x] = sum - mine;
    }
    __syncthreads();
    unsigned long long total = 0;   // a group's units
#pragma unroll
    for (int w = 0; w < WARPS; ++w) total += small.warp_units[w];
    // The list's W units in runs: each of them has `each` units, the first `more` one more.
    const unsigned long long W = total * groups;
    const unsigned runs = (unsigned)min((unsigned long long)(a.n_slots / a.step), W);
    const unsigned long long each = runs > 0 ? div64(W, runs) : 0;
    const unsigned more = (unsigned)(W - each * runs);
    auto run_from = [&](unsigned r) { return r >= runs ? W : each * r + min(r, more); };
    auto run_of = [&](unsigned long long unit) {
        const unsigned long long longer = (each + 1) * more;
        return (unsigned)(unit < longer ? div64(unit, each + 1) : more + div64(unit - longer, each));
    };
    if (run < runs) {
        unsigned long long u = run_from(run);
        const unsigned long long left = run_from(run + 1) - u;
        int group = 0;
        if (groups > 8) {
            group = (int)div64(u, total);
            u -= group * total;
        } else {
            for (; u >= total; ++group) u -= total;
        }
        // the last thread that has no more units before it
        int t = -1;
        unsigned long long before = 0, at = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const int n = __popc(__ballot_sync(0xffffffffu, before + small.units_before[32 * w + lane] <= u));
            if (n > 0) {
                t = 32 * w + n - 1;
                at = before + small.units_before[t];
            }
            before += small.warp_units[w];
        }
        u -= at;
        int seq = t * per;
        if (per > 1)   // and of its sequences
            for (; seq < pg.n_seq; seq += 32) {
                const unsigned own = seq + lane < pg.n_seq ? units_of<KT, PIECE_COST>(keys_of(pg, seq + lane)) : 0;
                unsigned sum = own;
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                    const unsigned up = __shfl_up_sync(0xffffffffu, sum, x);
                    if (lane >= x) sum += up;
                }
                const unsigned all = __shfl_sync(0xffffffffu, sum, 31);
                if (u >= all) {
                    u -= all;
                    continue;
                }
                const int n = __popc(__ballot_sync(0xffffffffu, sum <= u));   // of 32 that lie before
                u -= __shfl_sync(0xffffffffu, sum - own, n);
                seq += n;
                break;
            }
        start(ahead, pg, small.lengths, min(seq, pg.n_seq - 1), group, (int)u, left, lane);
    } else {
        start(ahead, pg, small.lengths, 0, 0, 0, 0, lane);
    }
    const bool by_pair = join_by_pair(a.H_kv, pg.n_seq, a.n_slots);
    const int g = lane >> 2, t4 = lane & 3;
    bool owner = false;

    // ---- tiles are asked for up to NS ahead, across pieces
    const uint32_t ring = smem_u32(sm) + warp * C::NS * C::STAGE;
    const int my_row = lane / C::CHUNKS, my_chunk = lane % C::CHUNKS;   // of each copy of RPL rows
    const uint32_t my_place = my_row * C::ROW + (swizzle<D>(my_row, my_chunk) << 4);
    const uint8_t *my_code = codes.k, *my_scale = codes.sk;              // row and chunk, key, from the pool's start on
    const int q_bytes = a.G * D * (DT == KVC_IN_F32 ? 4 : 2);            // a group's queries
    int ta = 0, ta_end = 0, keys = 0, chunk = 0;        // of the piece that tiles are asked for of
    int slot = -1, page_next = -1;                      // lane i's: of the i-th subtile from tile `chunk` on (-1: a hole); its
                                                        // page 16 tiles later, which is not looked at before
    bool rest_of_run;
    int stage_in = 0, stage_out = 0;
    uint32_t exists = 0;                                // lane s: a bit for each key of the tile in stage s
    auto page_of = [&](int tile, int seq) {
        const unsigned key = (unsigned)tile * KT + lane * 16;
        return key < (unsigned)keys ? __ldcg(pg.table + (int64_t)seq * pg.max_pages + key / (unsigned)pg.page_size) : -1;
    };
    auto slot_in = [&](int page, int tile) {
        return (unsigned)page < (unsigned)pg.n_pages ? page * pg.page_size + (int)(((unsigned)tile * KT + lane * 16) % (unsigned)pg.page_size) : -1;
    };
    auto begin_piece = [&]() {
        const Piece p = ahead->piece;
        const int h = p.h * a.step + member;
        ta = chunk = p.t0;
        ta_end = p.t1;
        keys = p.keys;
        const int page = page_of(chunk, p.seq);
        page_next = page_of(chunk + 16, p.seq);
        slot = slot_in(page, chunk);
        my_code = codes.k + my_row * codes.tok + h * codes.head + my_chunk * 16;
        my_scale = codes.sk + (lane & 15) * codes.s_tok + h * codes.s_head;
    };
    auto ask = [&]() {
        if (rest_of_run && ta >= ta_end) {
            rest_of_run = next(ahead, pg, small.lengths, groups, lane);
            if (rest_of_run) begin_piece();
        }
        if (rest_of_run) {
            if (ta - chunk == 16) {
                chunk = ta;
                slot = slot_in(page_next, chunk);
                page_next = page_of(chunk + 16, ahead->piece.seq);
            }
            const uint32_t kt = ring + stage_in * C::STAGE, place = kt + my_place;
            const int sl[2] = {__shfl_sync(0xffffffffu, slot, 2 * (ta - chunk)), __shfl_sync(0xffffffffu, slot, 2 * (ta - chunk) + 1)};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int bytes = sl[u] < 0 ? 0 : 16;
                const uint8_t *k = my_code + (uint64_t)(uint32_t)max(sl[u], 0) * codes.tok, *v = k + codes.v_from_k;
#pragma unroll
                for (int r = 0; r < 16; r += C::RPL) {
                    copy16(place + (16 * u + r) * C::ROW, k, bytes);
                    copy16(place + (16 * u + r) * C::ROW + C::TILE, v, bytes);
                    k += codes.rows;
                    v += codes.rows;
                }
            }
            const int mine = lane < 16 ? sl[0] : sl[1];   // a key for each lane: its scales
            const bool valid = mine >= 0 && lane < keys - ta * KT;
            const uint8_t *k = my_scale + (uint64_t)(uint32_t)max(mine, 0) * codes.s_tok;
            const uint32_t sc = kt + 2 * C::TILE + lane * C::NB * 2;
            copy_scales<C::NB * 2>(sc, k, valid);
            copy_scales<C::NB * 2>(sc + C::SC, k + codes.sv_from_sk, valid);
            const uint32_t all = __ballot_sync(0xffffffffu, valid);
            if (lane == stage_in) exists = all;
            stage_in = stage_in + 1 == C::NS ? 0 : stage_in + 1;
            ++ta;
        }
        copies_end_group();   // one for each call, so that the oldest is always NS - 1 before the newest
    };
    // the first piece's queries are on their way while its pages are looked up
    RawQueries<D, DT, NT> raw;
    auto read = [&]() {
        read_queries<D, DT, NT>(a.q + way->piece.seq * a.ld_q + (way->piece.h * a.step + member) * (int64_t)q_bytes, a.G, lane, raw);
    };
    constexpr bool EARLY = NT == 1 && DT != KVC_IN_F32;   // else the registers are not there
    bool some = rest_of_run = next(ahead, pg, small.lengths, groups, lane);
    for (int i = lane; i < (int)(sizeof(Way) / 4); i += 32) reinterpret_cast<int *>(way)[i] = reinterpret_cast<const int *>(ahead)[i];
    __syncwarp();
    if (EARLY && some) read();
    if (some) begin_piece();
    for (int i = 0; i < C::NS; ++i) ask();

    // sequences without keys have no unit in the list
    for (int i = blockIdx.x; i < pg.n_seq; i += gridDim.x) {
        if (keys_of(pg, i) > 0) continue;
        for (int e = threadIdx.x; e < a.H_q * D; e += THREADS) store_out<DT>(a.out, (int64_t)i * a.H_q * D + e, 0.f);
        if (a.lse)
            for (int e = threadIdx.x; e < a.H_q; e += THREADS) a.lse[(int64_t)i * a.H_q + e] = -INFINITY;
        if (by_pair)
            for (int e = threadIdx.x; e < a.H_kv; e += THREADS) a.desc[e * pg.n_seq + i] = make_int4(0, 0, 0, 0);
    }

    for (bool first = true; some; some = next(way, pg, small.lengths, groups, lane), first = false) {
        if (!EARLY || !first) read();
        uint32_t qf[D / 16][NT][2], eights[NT];
        float worth[NT][2];
        make_queries<D, DT, NT>(raw, a.scale_log2, lane, qf, eights, worth);
        float o[C::MT][NT][4], ob[C::NB][NT][4], m[NT][2], l[NT][2];
        __half2 factor[C::NB / 2];
#pragma unroll
        for (int i = 0; i < C::NB / 2; ++i) factor[i] = __float2half2_rn(0x1p15f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = NONE;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int b = 0; b < C::NB; ++b) ob[b][nt][0] = ob[b][nt][1] = ob[b][nt][2] = ob[b][nt][3] = 0.f;
#pragma unroll
            for (int i = 0; i < C::MT; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
        }
        for (int left = way->piece.t1 - way->piece.t0; left > 0; --left) {
            wait_groups_but<C::NS - 1>();
            __syncwarp();
            const uint32_t kt = ring + stage_out * C::STAGE, e = __shfl_sync(0xffffffffu, exists, stage_out);
#pragma unroll 1
            for (int u = 0; u < 2; u += C::U) {
                const uint32_t bits = C::U == 2 ? e : e >> (16 * u) & 0xFFFFu;
                if (bits != 0) attend<D, NT, C>(kt, 16 * u, bits, lane, qf, eights, worth, o, ob, m, l, factor);
            }
            if (left % FOLD == 0) fold_eights<NT, C>(o, ob);
            __syncwarp();   // before the stage is written again
            stage_out = stage_out + 1 == C::NS ? 0 : stage_out + 1;
            ask();
        }

        // ---- the piece is done
        fold_eights<NT, C>(o, ob);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
            }
        const Piece p = way->piece;
        const int h = p.h * a.step + member;
        const bool whole = p.t0 == 0 && p.t1 == p.nt;
        const int part = (c * 2 + (p.t0 == 0)) * a.G;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // this lane stores for one of its two heads, eight dimensions of each block, half of them its neighbour's
            const int head = nt * 8 + 2 * t4 + (g & 1);
            const float L = g & 1 ? l[nt][1] : l[nt][0], m_own = g & 1 ? m[nt][1] : m[nt][0];
            const float M = m_own == NONE ? -INFINITY : m_own;
            const float by = whole ? (L > 0.f || L != L ? 1.f / L : 0.f) : 1.f;
#pragma unroll
            for (int b = 0; b < C::NB; ++b) {
                const float w = 0x1p24f / __half2float(b & 1 ? __high2half(factor[b >> 1]) : __low2half(factor[b >> 1])) * by;
                float x[8];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float (&r)[4] = o[2 * b + (n >> 1)][nt];
                    const float e0 = n & 1 ? r[2] * 0.0625f : r[0], e1 = n & 1 ? r[3] * 0.0625f : r[1];
                    const float got = __shfl_xor_sync(0xffffffffu, g & 1 ? e0 : e1, 4);
                    x[2 * n] = (g & 1 ? got : e0) * w;
                    x[2 * n + 1] = (g & 1 ? e1 : got) * w;
                }
                const int dim = 32 * b + 8 * (g >> 1);
                if (head >= a.G) continue;
                if (whole) store_out8<DT>(a.out, ((int64_t)p.seq * a.H_q + h * a.G + head) * D + dim, x);
                else store_out8<KVC_IN_F32>(a.part_o, (int64_t)(part + head) * D + dim, x);
            }
            if (g < 2 && head < a.G) {
                if (!whole)   // the join passes over parts with M = -infinity, but a NaN has to reach it
                    a.part_ml[part + head] = make_float2(isnan(L) ? INFINITY : M, L);
                else if (a.lse)
                    a.lse[(int64_t)p.seq * a.H_q + h * a.G + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
            }
        }
        if (p.t0 == 0 && (by_pair || !whole)) {
            owner = true;
            if (lane == 0) {
                // the run that holds the pair's last unit
                const int last = whole ? 0 : (int)run_of(run_from(run + 1) + (p.nt - p.t1) - 1);
                a.desc[by_pair ? h * pg.n_seq + p.seq : c] = make_int4(p.seq, h, whole ? 0 : last - (int)run + 1, c);
            }
        }
    }
    if (!by_pair && !owner && lane == 0) a.desc[c] = make_int4(0, 0, 0, 0);
}

template <int D, int DT, int NT>
int launch_t(const PagedView &pg, const Args &a, const Codes &codes, cudaStream_t s) {
    using C = Cfg<D, DT, NT>;
    if (allow_dynamic_smem((const void *)decode_paged_q4_kernel<D, DT, NT>, C::SMEM) != KVC_OK) return KVC_ECUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.n_slots / WARPS);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, decode_paged_q4_kernel<D, DT, NT>, pg, a, codes) != cudaSuccess) return KVC_ECUDA;
    // The join: warps' runs make four times as many partials as CTAs' would, and starting threads is most of what it costs.  A
    // CTA gets as many threads as a pair will have partials for, if all CTAs then fit the GPU at once.  With 64, 128, 256
    // and 512 threads, in us: the 96 sequences 53.5, 53.7, 55.7 and 61.9 (of 700 tokens 27.6, 28.5, 32.3 and 40.4), eight 15.7,
    // 14.4, 13.8 and 14.2, one of 58,300 34.0, 28.4, 23.6 and 23.3 (22.4 with eight partials loaded together).  Joins by slot, 400
    // sequences of 700: a CTA of 256 for each 82, for two 84, for four 95; of 128 for each 86.
    void (*join)(const Args, int) = combine_paged_kernel<D, DT, true>;
    cfg.gridDim = dim3(a.n_slots);
    cfg.blockDim = dim3(COMBINE_THREADS);
    cfg.dynamicSmemBytes = 0;
    int joins = a.n_slots;
    if (join_by_pair(a.H_kv, pg.n_seq, a.n_slots)) {
        joins = a.H_kv * pg.n_seq;   // n_slots at most
        const int parts = min(a.n_slots / joins, (pg.max_pages * pg.page_size - 1) / KT + 1) + 1;
        auto fits = [&](int threads) {
            return threads / (D / 4) <= parts && (int64_t)joins * a.G * threads <= 2048 * (int64_t)sm_count();
        };
        constexpr int MOST = 64;   // partials that 256 threads join as fast
        const int threads = parts > MOST && fits(512) ? 512 : fits(256) ? 256 : fits(128) ? 128 : 64;
        join = threads == 512   ? combine_paged_kernel<D, DT, false, 512, 8>
               : threads == 256 ? combine_paged_kernel<D, DT, false, 256>
               : threads == 128 ? combine_paged_kernel<D, DT, false, 128>
                                : combine_paged_kernel<D, DT, false, 64>;
        cfg.gridDim = dim3(joins, a.G);
        cfg.blockDim = dim3(threads);
    }
    if (cudaLaunchKernelEx(&cfg, join, a, joins) != cudaSuccess) return KVC_ECUDA;
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ECUDA;
}

template <int D>
int launch_d(int dtype, const PagedView &pg, const Args &a, const Codes &codes, cudaStream_t s) {
    switch (dtype) {
#define KVC_CASE(DT)                                                                             \
    case DT:                                                                                     \
        return a.G <= 8 ? launch_t<D, DT, 1>(pg, a, codes, s) : launch_t<D, DT, 2>(pg, a, codes, s);
        KVC_CASE(KVC_IN_F32)
        KVC_CASE(KVC_IN_BF16)
        KVC_CASE(KVC_IN_F16)
#undef KVC_CASE
        default: return KVC_EINVAL;
    }
}

}  // namespace

int paged_q4_slots(int G) { return WARPS * ctas_per_sm(G <= 8 ? 1 : 2) * sm_count(); }

int launch_decode_paged_q4(const kvc_cache &c, const kvc_pages &p, int layer, int dtype, const paged::Args &args, cudaStream_t s) {
    const Geom g = geom_of(c.d);
    Args a = args;
    a.step = c.d.n_head_kv % 4 == 0 ? 4 : c.d.n_head_kv % 2 == 0 ? 2 : 1;
    const int64_t code = layer * g.c_layer / 2, scale = layer * g.s_layer * 2;
    const uint8_t *k = static_cast<const uint8_t *>(c.k_q), *v = static_cast<const uint8_t *>(c.v_q);
    const uint8_t *sk = static_cast<const uint8_t *>(c.k_s), *sv = static_cast<const uint8_t *>(c.v_s);
    const Codes codes = {k + code, sk + scale, v - k, sv - sk, g.c_head / 2, g.s_head * 2, (uint32_t)(g.c_tok / 2),
                         (uint32_t)(g.c_tok / 2 * (1024 / c.d.head_dim)), (uint32_t)(g.s_tok * 2)};
    const PagedView pg = paged_view(c, p);
    return c.d.head_dim == 128 ? launch_d<128>(dtype, pg, a, codes, s) : launch_d<64>(dtype, pg, a, codes, s);
}

}  // namespace kvc
