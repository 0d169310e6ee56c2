// Attention of one new token for each sequence over a paged pool.
//
//   out[i][h] = sum_{j < len[i]} softmax_j(q[i][h] . khat[j][h/G] / sqrt(D)) vhat[j][h/G]
//
// What bounds it: every key and value is read once and used for the G query heads of its group, so the floor
// is the pool's bytes over the HBM rate (a few operations per byte; q8_0 also has to turn each code into fp16).
//
// Work split.  The keys of all (kv head, sequence) pairs, in tiles of 64 and with a charge for each pair, form
// one list that is cut into equal runs, one for each CTA (two or three per SM), wherever the boundaries fall: ragged
// lengths, one long sequence and many short ones all fill the GPU.  Heads are outermost, so where their number
// divides the CTAs' the CTAs of all heads pass the same tokens at the same time, which is what a layer-major
// pool (a token's heads side by side) wants of DRAM and L2.  The lengths are read on the device.  A pair inside one
// run is written straight to out; a pair cut by run boundaries leaves one partial (O, maximum, sum) per run in
// scratch - at most two per CTA - and a second kernel joins them in run order.
//
// One CTA: a producer warp looks up the pages and keeps a ring of tiles in flight by TMA (one box per page piece,
// swizzled so that both products read them without bank conflicts, scales by 8-byte asynchronous copies); four
// consumer warps take 16 keys of each tile, one subtile each, which always lies within one page.  A warp keeps its own
// reference, 2^7 below the running maximum (raised only when a score passes that by 2^8, so that the accumulators are seldom
// rescaled), and sum, and the four are joined when a pair ends.  Both products run on warp-level matrix instructions with
// the keys (S^T = K Q^T) and the value dimensions (O^T = V^T P^T) as the 16-row side, so that a group of up
// to 8 query heads wastes nothing but padding columns:
//   - the order of dimensions in the first product and of keys in both is free as long as the operands agree,
//     so each lane loads 8 or 16 consecutive bytes of a row, and codes need no shuffles between lanes;
//   - q8_0 codes enter the first product as the integers they are; each block's products are scaled by d in
//     float32.  In the second product the values are fp16(d * q) and the numerators p are rounded to fp16, in two parts
//     where the output is finer than bf16;
//   - S^T leaves the first product with a lane per key and enters the second with a lane per head: one 8x8
//     transposition for each half of the subtile.
// Keys past the length and pages outside the pool are never loaded, or are given zero weight and zeroed values.
//
// Measured (40 query heads, 8 kv heads of 128; of the rate of a copy): 96 sequences of 5 to 16,384 tokens, q8_0 pool, to an
// fp16 output 82 us (4.9 TB/s, 0.73), to bf16 79 to 81, in 16 heads to a group 124; f16 pool 120 to 122 us (6.3 TB/s, 0.92);
// one sequence of 58,300, q8_0, 30 us (4.2 TB/s, 0.62); eight of about 2,100, f16, 18.7 us (3.7 TB/s, 0.55).  The last two
// pay about 7 us (a sequence of 64 tokens) for the two launches, the list, the first loads and the join; q8_0 pools are
// bound by the consumers' chains of loads, conversions and products.
// Every mbarrier wait is bounded (2 s); a wait that gives up sets the device status word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace kvc {

namespace {

// set by a kernel of this translation unit that gave up a bounded wait (read and cleared with the other kernels' status)
__device__ int g_paged_status;

using namespace ptx;

constexpr int CW = 4;               // consumer warps, 16 keys of a tile each (of q4_0: SUBS * 16)
constexpr int THREADS = 32 * (CW + 1);
// CTAs per SM: two, whose consumers keep up with the loads of an f16 pool; three for q8_0, where they do not, but for groups
// of more than 8 query heads (NT = 2), whose accumulators three leave too few registers.  With three and two, in us (bf16, 8
// kv heads, back to back): up to 8 heads to a group, D = 128 the 96 sequences below 79 and 83, one of 58,300 31.7 and 32.2, 96
// of 700 40.9 and 38.1; D = 64 68 and 69, 21.6 and 25.5.  16 heads, D = 128 144 and 125, 50 and 43; D = 64 70 and 73: there
// two are 5% slower.
constexpr int ctas_per_sm(int ct, int NT) { return ct != KVC_F16 && NT == 1 ? 3 : 2; }
constexpr int smem_budget(int ct, int NT) { return ctas_per_sm(ct, NT) == 3 ? 76800 : 115712; }   // 75 and 113 KB
// Subtiles of 16 keys that a consumer warp takes of a tile.
constexpr int subs_of(int ct) { return ct == KVC_Q4_0 ? 2 : 1; }
constexpr int keys_per_tile(int ct) { return CW * 16 * subs_of(ct); }
constexpr int COMBINE_THREADS = 256;
constexpr int MAX_NS = 10;          // tiles of the longest ring (16 heads of 64, q8_0)
// What starting and ending a pair costs, in tiles.  With 0, 1, 2 and 4, in us (q8_0, bf16): 96 sequences of 5 to 16,384 91, 85,
// 79 and 87, in 16 heads to a group 136, 131, 125 and 112, with D = 64 61, 57, 68 and 72, f16 123, 119, 120 and 120; 170 sequences
// of 10 to 3,000, 2 kv heads 25, 20, 19 and 21; one of 58,300 31.4, 31.4, 31.7 and 31.6.  (The cuts' places, and with them
// which CTAs pass the same tokens together, move with it.)
constexpr int PIECE_COST = 2;
// A row's reference lies SHIFT_LOG2 below its greatest score, so that the numerators are 2^7 there (2^15 at most before the
// reference is raised) and fp16 holds them down to 2^-31 of it.  With the reference at the score itself those below 2^-25
// vanished from O, but not from the sum: long contexts lost them.
constexpr float SHIFT_LOG2 = 7.0f, RESCALE_LOG2 = SHIFT_LOG2 + 8.0f;
constexpr float LN2 = 0.69314718055994531f;

template <int D, int CT, int DT, int NT>
struct Cfg {
    static constexpr bool Q8 = CT == KVC_Q8_0, Q4 = CT == KVC_Q4_0, SCALES = Q8 || Q4;
    static constexpr int SUBS = subs_of(CT), KT = keys_per_tile(CT);

    // Both operands of a q8_0 pool's second product are rounded to fp16, which an fp16 or float32 output shows (the 96
    // sequences above: 1.53 times the error of the output's own rounding): there the numerators enter in two parts, for 4%
    // of the time (1.41 times).  A bf16 output's rounding, eight times as coarse, hides it.
    static constexpr bool FINE = Q8 && DT != KVC_IN_BF16;
    static constexpr int NB = D / 32;                       // q8_0 blocks per row
    static constexpr int ROW = Q4 ? D / 2 : D * (Q8 ? 1 : 2);   // bytes of a row
    static constexpr int TILE = KT * ROW;                   // a K or V tile
    static constexpr int SC = SCALES ? KT * NB * 2 : 0;         // a tile's scales
    static constexpr int STAGE = 2 * TILE + ((2 * SC + 1023) & ~1023);
    static constexpr int MT = D / 16;                       // 16-row tiles of O^T
    static constexpr int OWN = MT / CW;                     // of which each warp writes
    static constexpr int RED = MT * NT * (CW - 1) * 512;    // the other warps' accumulators
    static constexpr int ESZ = DT == KVC_IN_F32 ? 4 : 2;
    static constexpr int QB = 8 * NT * D * ESZ;             // the most that a group's queries take
    static constexpr int MISC = 1024;
    static constexpr int FIT = (smem_budget(CT, NT) - 1024 - RED - QB - MISC) / STAGE;
    static constexpr int NS = FIT < MAX_NS ? FIT : MAX_NS;
    static constexpr int OFF_RED = NS * STAGE, OFF_MISC = OFF_RED + RED, OFF_Q = OFF_MISC + MISC;
    static constexpr int Q_ROOM = smem_budget(CT, NT) - 1024 - OFF_Q;
    static_assert(NS >= 2 && Q_ROOM >= QB, "shared memory plan");
};
constexpr int MAX_NQ = 4;           // slots for the queries of pieces to come: as many as fit (1, 2 and 4 take the same time)

// what the small area behind the ring holds
struct Misc {
    uint64_t full[MAX_NS], empty[MAX_NS], q_full[MAX_NQ], q_empty[MAX_NQ], stall;
    uint8_t count[MAX_NS][2 * CW];       // keys of each subtile that exist
    float2 ml[CW][16];                   // reference and sum of each warp and head
    unsigned long long warp_units[CW + 1], total;
    uint32_t tiles, queries;             // what the producer has asked for in all
    int first_seq, rest, abort;
};
static_assert(sizeof(Misc) <= 1024, "small area");

}  // namespace

struct DecodePagedArgs {
    const uint16_t *ks, *vs;             // scales of the layer
    int64_t s_tok, s_head;
    const uint8_t *q;
    int64_t ld_q;                        // bytes
    void *out;
    float *lse;
    float *part_o;                       // [CTA][2][G][D]
    float2 *part_ml;                     // [CTA][2][G]
    int4 *desc;                          // [join]: sequence, kv head, partials (0: none), CTA that begins the pair
    int H_q, H_kv, G, box, n_slots, n_q;
    float scale_log2;
    uint64_t stall_ns;                   // test hook: > 0 makes the first consumer warp wait for what never comes
};

// A q4_0 pool's kernels, a translation unit of their own.
int launch_decode_paged_q4(const kvc_cache &c, int layer, int page_size, int dtype, const PagedView &pg,
                           const DecodePagedArgs &a, cudaStream_t s);
int read_and_clear_paged_q4_status(int32_t *status);

namespace {

using Args = DecodePagedArgs;

// A pair's keys, or the part of them that falls into one CTA's run.
struct Piece {
    int seq, h, t0, t1, nt, keys;
};

__device__ __forceinline__ int keys_of(const PagedView &pg, int i) {
    return min(max(__ldcg(pg.len + i), 0), pg.max_pages * pg.page_size);
}
// One join for each pair where there are no more pairs than CTAs, else one for each CTA: the pair that it begins and
// others finish, if there is one.  (A join without work costs a block of each query head: one sequence of 58,300 tokens
// takes 1.4 us less than with a join for each CTA.)
__host__ __device__ __forceinline__ bool join_by_pair(int H_kv, int n_seq, int n_slots) {
    return (int64_t)H_kv * n_seq <= n_slots;
}
template <int KT>
__device__ __forceinline__ int tiles_of(int keys) { return (keys + KT - 1) / KT; }
template <int KT>
__device__ __forceinline__ int units_of(int keys) { return keys > 0 ? tiles_of<KT>(keys) + PIECE_COST : 0; }

// A warp's way through its CTA's run of the list: kv heads, in each the sequences, in each its units.  The
// lengths of 32 sequences are held a lane each, so that most steps load nothing.
template <int KT>
struct Walk {
    int seq, h, x, base, held;   // x: units of the current pair that lie before this run
    unsigned long long left;
    __device__ __forceinline__ Walk(const PagedView &pg, int seq_, int h_, int x_, unsigned long long left_)
        : seq(seq_), h(h_), x(x_), left(left_) { load(pg); }
    __device__ __forceinline__ void load(const PagedView &pg) {
        base = seq;
        const int i = base + (threadIdx.x & 31);
        held = i < pg.n_seq ? keys_of(pg, i) : 0;
    }
    __device__ __forceinline__ bool next(const PagedView &pg, int H_kv, Piece &p) {
        while (left > 0 && h < H_kv) {
            if (seq - base >= 32 || seq < base) load(pg);
            const int keys = __shfl_sync(0xffffffffu, held, seq - base), all = units_of<KT>(keys);
            const int x1 = (int)min((unsigned long long)all, x + left);
            p = {seq, h, max(x - PIECE_COST, 0), max(x1 - PIECE_COST, 0), tiles_of<KT>(keys), keys};
            left -= x1 - x;
            x = 0;
            if (++seq == pg.n_seq) { seq = 0; ++h; }
            if (p.t1 > p.t0) return true;
        }
        return false;
    }
};

// The list of W units is cut into P runs, [W c / P, W (c + 1) / P), none of them empty: one for each CTA, or W.
__device__ __forceinline__ unsigned long long runs_of(unsigned long long W) {
    return min((unsigned long long)gridDim.x, W);
}
__device__ __forceinline__ unsigned long long run_start(unsigned long long W, unsigned c) {
    const unsigned long long P = runs_of(W);
    return c >= P ? W : W * c / P;
}

// A wait of a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          uint64_t limit_ns = 2000000000ull) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit_ns));
}

template <int DT>
__device__ __forceinline__ void store_out(void *out, int64_t i, float x) {
    if constexpr (DT == KVC_IN_F32) static_cast<float *>(out)[i] = x;
    else if constexpr (DT == KVC_IN_BF16) static_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(x);
    else static_cast<__half *>(out)[i] = __float2half_rn(x);
}

// the order of the eight keys of half a subtile: rows 2i and 2i+1 differ in bit 2, even rows (and odd rows) in bits
// 1 and 2, which is what makes every swizzled read below free of bank conflicts (a row of 128 bytes)
__device__ __forceinline__ int key_of(int r) { return r ^ ((r & 1) << 2); }

__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
// bytes c ^ 0x80 under the high byte 0x64 are the fp16 numbers 1152 + c
__device__ __forceinline__ uint32_t unbias(uint32_t u) { return as_u32(__hsub2(as_half2(u), as_half2(0x64806480u))); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}

// ---- q4_0 ------------------------------------------------------------------------------------------------------
// A nibble n (code + 8) that stays where it lies in the low byte of a half is the fp16 subnormal n 2^-24 or n 2^-20: an AND
// with 0x000F000F or 0x00F000F0 makes two operands of a product, exactly, and no subtraction or conversion is left
// to do for each value.  What the places are worth and the 8 are taken care of outside of the loops over values:
//   - first product: the queries of the lower nibbles are 16 times as large, and a block's accumulators begin at -8
//     times the sum of its queries;
//   - second product: V's scales are multiplied into the numerators (in float32, before their one rounding), so the values
//     are the nibbles; a further row of eights in place of them sums the 8 of all, which is subtracted at the end.
// So that numerators times scales stay in fp16's range, a row's reference includes the greatest scale of V that the warp
// has met (d_log2), and it is raised when a greater one appears.

template <int DT>
__device__ __forceinline__ void q4_load_q(uint32_t at, float (&v)[8]) {
    const uint4 x = lds128(at);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (DT == KVC_IN_F32) {
        const uint4 y = lds128(at + 16);
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
// magnitude from 2^-100 to 2^100 keeps its 11 bits.  c0: where the accumulators of a block begin for this lane's two
// columns, worth: what their products are worth in powers of two.
template <int D, int DT, int NT>
__device__ __forceinline__ void q4_queries(uint32_t q_at, int G, float scale_log2, int lane, uint32_t (&qf)[D / 16][NT][2],
                                           float (&c0)[D / 32][NT][2], float (&worth)[NT][2]) {
    const int g = lane >> 2, t4 = lane & 3;
    constexpr int ESZ = DT == KVC_IN_F32 ? 4 : 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int head = nt * 8 + g;
        float most = 0.f, v[8];
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            if (head < G) {
                q4_load_q<DT>(q_at + (head * D + 32 * b + 8 * t4) * ESZ, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
            }
        }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const int ex = most > 0.f ? min(max((int)(__float_as_uint(most) >> 23) - 127, -100), 100) : 0;
        const float lo = __uint_as_float((uint32_t)(127 + 10 - ex) << 23), hi = 16.f * lo;
        const float w = __uint_as_float((uint32_t)(127 + 10 + ex) << 23) * scale_log2;
#pragma unroll
        for (int e = 0; e < 2; ++e) worth[nt][e] = __shfl_sync(0xffffffffu, w, (2 * t4 + e) * 4);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
            if (head < G) q4_load_q<DT>(q_at + (head * D + 32 * b + 8 * t4) * ESZ, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t p = pack_half2(v[2 * i] * (i & 1 ? lo : hi), v[2 * i + 1] * (i & 1 ? lo : hi));
                const float2 f = __half22float2(as_half2(p));
                sum += (f.x + f.y) * (i & 1 ? 1.f : 0.0625f);
                qf[2 * b + (i >> 1)][nt][i & 1] = p;
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            sum *= -0x1p-17f;   // eight of the upper nibbles' units
#pragma unroll
            for (int e = 0; e < 2; ++e) c0[b][nt][e] = __shfl_sync(0xffffffffu, sum, (2 * t4 + e) * 4);
        }
    }
}

// A warp's keys of one tile: scores, numerators, sums.
template <int D, int NT, class C>
__device__ __forceinline__ void q4_tile(uint32_t kt, const uint8_t *counts, int warp, int lane, const uint32_t (&qf)[D / 16][NT][2],
                                        const float (&c0)[C::NB][NT][2], const float (&worth)[NT][2], float (&o)[C::MT][NT][4],
                                        float (&ob)[C::NB][NT][4], float (&m)[NT][2], float (&l)[NT][2], __half2 &d_most,
                                        float &d_log2) {
    constexpr int U = C::SUBS, NB = C::NB;
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
    int count[U], any = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) any |= count[u] = counts[u];
    if (any == 0) return;
    const uint32_t vt = kt + C::TILE, sc = vt + C::TILE;
    const int g = lane >> 2, t4 = lane & 3;
    // ldmatrix: lane i names row i % 8 of matrix i / 8: keys 0 to 7 and 8 to 15 of a block (16 bytes), then of the next one
    const int mrow = (lane & 7) + 8 * ((lane >> 3) & 1), mchunk = lane >> 4;
    auto at = [&](uint32_t tile, int u, int b) {   // swizzled as the TMA wrote it (rows of 64 or 32 bytes)
        const int row = (warp * U + u) * 16 + mrow, c = b + mchunk;
        return tile + row * C::ROW + ((D == 128 ? c ^ ((mrow >> 1) & 3) : c ^ ((mrow >> 2) & 1)) << 4);
    };
    auto scales = [&](uint32_t base, int u, int half, __half2 (&d)[NB / 2]) {
        const uint32_t p = base + ((warp * U + u) * 16 + g + 8 * half) * (2 * NB);
        if constexpr (NB == 4) {
            const uint2 x = lds64(p);
            d[0] = as_half2(x.x); d[1] = as_half2(x.y);
        } else {
            d[0] = as_half2(lds32(p));
        }
    };
    float s[U][NT][4];
    __half2 dv[U][2][NB / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        __half2 dk[2][NB / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            scales(sc, u, h, dk[h]);
            scales(sc + C::SC, u, h, dv[u][h]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
            uint32_t w[4];
            ldmatrix_x4(w, at(kt, u, b));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t ka = w[2 * x], kb = w[2 * x + 1], ka8 = ka >> 8, kb8 = kb >> 8;
                const uint32_t A[4] = {ka & LO, kb & LO, ka & HI, kb & HI}, B[4] = {ka8 & LO, kb8 & LO, ka8 & HI, kb8 & HI};
                const float2 f = __half22float2(dk[0][b >> 1]), h = __half22float2(dk[1][b >> 1]);
                const float ca = x ? f.y : f.x, cb = x ? h.y : h.x;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float acc[4] = {c0[b + x][nt][0], c0[b + x][nt][1], c0[b + x][nt][0], c0[b + x][nt][1]};
                    mma_16816(acc, A, qf[2 * (b + x)][nt][0], qf[2 * (b + x)][nt][1]);
                    mma_16816(acc, B, qf[2 * (b + x) + 1][nt][0], qf[2 * (b + x) + 1][nt][1]);
                    s[u][nt][0] = fmaf(acc[0], ca, s[u][nt][0]);
                    s[u][nt][1] = fmaf(acc[1], ca, s[u][nt][1]);
                    s[u][nt][2] = fmaf(acc[2], cb, s[u][nt][2]);
                    s[u][nt][3] = fmaf(acc[3], cb, s[u][nt][3]);
                }
            }
        }
        if (count[u] < 16) {   // the last subtile of a sequence, or one of a hole
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (g >= count[u]) s[u][nt][0] = s[u][nt][1] = -INFINITY;
                if (g + 8 >= count[u]) s[u][nt][2] = s[u][nt][3] = -INFINITY;
            }
        }
    }
    __half2 d_here = __float2half2_rn(0.f);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) d_here = __hmax2(d_here, __habs2(dv[u][h][i]));
    bool above = !__hble2(d_here, d_most);
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[nt][e] = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
#pragma unroll
            for (int u = 1; u < U; ++u) top[nt][e] = fmax3(top[nt][e], s[u][nt][e], s[u][nt][e + 2]);
            above |= fmaf(top[nt][e], worth[nt][e], d_log2) > m[nt][e] + RESCALE_LOG2;
        }
    if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1)
            d_here = __hmax2(d_here, as_half2(__shfl_xor_sync(0xffffffffu, as_u32(d_here), x)));
        const float d = fmaxf(__half2float(__low2half(d_most)),
                              fmaxf(__half2float(__low2half(d_here)), __half2float(__high2half(d_here))));
        d_most = __float2half2_rn(d);
        d_log2 = d > 0.f ? (float)((int)(__float_as_uint(d) >> 23) - 126) : 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = top[nt][e];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                const float m_new = fmaxf(m[nt][e], fmaf(x, worth[nt][e], d_log2 - SHIFT_LOG2));
                f[e] = m[nt][e] == m_new ? 1.f : ex2(m[nt][e] - m_new);
                m[nt][e] = m_new;
                l[nt][e] *= f[e];
            }
#pragma unroll
            for (int i = 0; i < C::MT; ++i) {
                o[i][nt][0] *= f[0]; o[i][nt][1] *= f[1]; o[i][nt][2] *= f[0]; o[i][nt][3] *= f[1];
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                ob[i][nt][0] *= f[0]; ob[i][nt][1] *= f[1]; ob[i][nt][2] *= f[0]; ob[i][nt][3] *= f[1];
            }
        }
    }
    float ref[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) ref[nt][e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][nt][i] = ex2(fmaf(s[u][nt][i], worth[nt][i & 1], -ref[nt][i & 1]));
            l[nt][0] += s[u][nt][0] + s[u][nt][2];
            l[nt][1] += s[u][nt][1] + s[u][nt][3];
        }
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
            uint32_t w[4];
            ldmatrix_x4_trans(w, at(vt, u, b));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t va = w[2 * x], vb = w[2 * x + 1], va8 = va >> 8, vb8 = vb >> 8;
                const uint32_t A[4] = {va & LO, va & HI, vb & LO, vb & HI}, B[4] = {va8 & LO, va8 & HI, vb8 & LO, vb8 & HI};
                const uint32_t E[4] = {0x00800080u, 0x00800080u, 0x00800080u, 0x00800080u};   // eights as upper nibbles
                const float2 f = __half22float2(dv[u][0][b >> 1]), h = __half22float2(dv[u][1][b >> 1]);
                const float ca = x ? f.y : f.x, cb = x ? h.y : h.x;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t p0 = movmatrix_trans(pack_half2(s[u][nt][0] * ca, s[u][nt][1] * ca));
                    const uint32_t p1 = movmatrix_trans(pack_half2(s[u][nt][2] * cb, s[u][nt][3] * cb));
                    mma_16816(o[2 * (b + x)][nt], A, p0, p1);
                    mma_16816(o[2 * (b + x) + 1][nt], B, p0, p1);
                    mma_16816(ob[b + x][nt], E, p0, p1);
                }
            }
        }
    }
}

template <int D, int CT, int DT, int NT>
__global__ void __launch_bounds__(THREADS, ctas_per_sm(CT, NT))
    decode_paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const PagedView pg, const Args a) {
    using C = Cfg<D, CT, DT, NT>;
    constexpr bool Q8 = C::Q8, Q4 = C::Q4;
    constexpr int KT = C::KT, SUBS = C::SUBS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    Misc *ms = reinterpret_cast<Misc *>(sm + C::OFF_MISC);
    volatile int *s_abort = &ms->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ms->abort = 0;
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&ms->full[s], C::SCALES ? 33 : 1);
            mbar_init(&ms->empty[s], CW);
        }
        for (int s = 0; s < MAX_NQ; ++s) {
            mbar_init(&ms->q_full[s], 1);
            mbar_init(&ms->q_empty[s], CW);
        }
        mbar_init(&ms->stall, 1);
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    // ---- this CTA's run of the list: where it starts
    {
        const int per = (pg.n_seq + THREADS - 1) / THREADS;
        const int i0 = min((int)threadIdx.x * per, pg.n_seq), i1 = min(i0 + per, pg.n_seq);
        unsigned long long mine = 0;
        for (int i = i0; i < i1; ++i) mine += units_of<KT>(keys_of(pg, i));
        unsigned long long sum = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const unsigned long long up = __shfl_up_sync(0xffffffffu, sum, x);
            if (lane >= x) sum += up;
        }
        if (lane == 31) ms->warp_units[warp] = sum;
        __syncthreads();
        unsigned long long before = sum - mine, total = 0;
        for (int w = 0; w <= CW; ++w) {
            if (w < warp) before += ms->warp_units[w];
            total += ms->warp_units[w];
        }
        unsigned long long r = total ? run_start(total * a.H_kv, blockIdx.x) % total : 0;
        if (threadIdx.x == 0) ms->total = total;
        if (r >= before && r < before + mine) {
            r -= before;
            int i = i0;
            for (; i + 1 < i1; ++i) {
                const unsigned long long n = units_of<KT>(keys_of(pg, i));
                if (r < n) break;
                r -= n;
            }
            ms->first_seq = i;
            ms->rest = (int)r;
        }
        __syncthreads();
    }
    const unsigned long long W = ms->total * a.H_kv, u0 = run_start(W, blockIdx.x), u1 = run_start(W, blockIdx.x + 1);
    Walk<KT> walk(pg, u1 > u0 ? ms->first_seq : 0, u1 > u0 ? (int)(u0 / ms->total) : 0, u1 > u0 ? ms->rest : 0, u1 - u0);

    if (warp == CW) {
        // ------------------------------------------------------------------ producer
        // Tiles are taken eight (of q4_0 four) at a time, across pieces: lane PER i + j knows subtile j of the i-th.  The
        // pages of the next ones are being looked up while these are copied.
        constexpr int PER = KT / 16, BATCH = 32 / PER;
        struct Batch {
            int n, seq, h, t, keys, page;
            bool first;
        };
        uint32_t n = 0, nq = 0;
        bool more = true;
        Piece p = {0, 0, 0, 0, 0, 0};
        int t = 0;
        auto take = [&](Batch &b) {
            b.n = 0;
            b.keys = 0;
            b.t = 0;
            while (b.n < BATCH && more) {
                const bool first = t >= p.t1;
                if (first) {
                    more = walk.next(pg, a.H_kv, p);
                    if (!more) break;
                    t = p.t0;
                }
                if (lane / PER == b.n) {
                    b.seq = p.seq; b.h = p.h; b.t = t; b.keys = p.keys; b.first = first;
                }
                ++t;
                ++b.n;
            }
            const int key = b.t * KT + lane % PER * 16;
            b.page = key < b.keys ? __ldcg(pg.table + (int64_t)b.seq * pg.max_pages + key / pg.page_size) : -1;
        };
        if (lane == 0) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        const int q_bytes = a.G * D * C::ESZ, per_box = a.box >> 4, boxes = KT / a.box;
        Batch cur, nxt;
        take(cur);
        for (bool ok = true; ok && cur.n > 0; cur = nxt) {
            take(nxt);
            const int key0 = cur.t * KT + lane % PER * 16;
            // my subtile's first pool position (-1: none of its keys exist) and how many of its keys exist
            const int slot = (unsigned)cur.page < (unsigned)pg.n_pages ? cur.page * pg.page_size + key0 % pg.page_size : -1;
            const int count = slot < 0 ? 0 : min(16, cur.keys - key0);
            for (int i = 0; i < cur.n; ++i) {
                const int h = __shfl_sync(0xffffffffu, cur.h, PER * i);
                if (__shfl_sync(0xffffffffu, (int)cur.first, PER * i)) {
                    const int qs = nq % a.n_q, seq = __shfl_sync(0xffffffffu, cur.seq, PER * i);
                    if (nq >= (uint32_t)a.n_q && !warp_wait(&ms->q_empty[qs], ((nq / a.n_q) - 1) & 1, s_abort)) { ok = false; break; }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&ms->q_full[qs], q_bytes);
                        bulk_load(sm + C::OFF_Q + qs * q_bytes, a.q + seq * a.ld_q + (int64_t)h * q_bytes, q_bytes, &ms->q_full[qs]);
                    }
                    ++nq;
                }
                const int st = n % C::NS;
                if (n >= (uint32_t)C::NS && !warp_wait(&ms->empty[st], ((n / C::NS) - 1) & 1, s_abort)) { ok = false; break; }
                uint8_t *kt = sm + st * C::STAGE, *vt = kt + C::TILE;
                if (lane / PER == i) ms->count[st][lane % PER] = count;
                const int box_slot = __shfl_sync(0xffffffffu, slot, PER * i + lane * per_box % PER);
                const bool load = lane < boxes && box_slot >= 0;
                const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
                __syncwarp();   // the counts before the arrival that publishes them (shuffles and ballots order no memory)
                if (lane == 0) mbar_arrive_expect_tx(&ms->full[st], loads * 2 * a.box * C::ROW);
                __syncwarp();
                if (load) {
                    const int off = lane * a.box * (C::SCALES ? C::ROW : 128);
#pragma unroll
                    for (int hh = 0; hh < (C::SCALES ? 1 : D / 64); ++hh) {
                        tma_load_3d(kt + hh * KT * 128 + off, &tm_k, &ms->full[st], hh * 64, box_slot, h);
                        tma_load_3d(vt + hh * KT * 128 + off, &tm_v, &ms->full[st], hh * 64, box_slot, h);
                    }
                }
                if constexpr (C::SCALES) {
                    uint8_t *sc = vt + C::TILE;
#pragma unroll
                    for (int x = 0; x < 2 * KT / 32; ++x) {
                        const int key = (x * 32 + lane) & (KT - 1), is_v = x / (KT / 32);
                        const int sl = __shfl_sync(0xffffffffu, slot, PER * i + (key >> 4));
                        const bool valid = (key & 15) < __shfl_sync(0xffffffffu, count, PER * i + (key >> 4));
                        const uint16_t *src = (is_v ? a.vs : a.ks) + (valid ? (int64_t)(sl + (key & 15)) * a.s_tok + h * a.s_head : 0);
                        cp_async_zfill<C::NB * 2>(sc + is_v * C::SC + key * C::NB * 2, src, valid);
                    }
                    cp_async_arrive(&ms->full[st]);
                }
                ++n;
            }
        }
        if (lane == 0) {
            ms->tiles = n;
            ms->queries = nq;
        }
    } else {
        // ------------------------------------------------------------------ consumers
        const int g = lane >> 2, t4 = lane & 3;
        const int kp = key_of(g);                               // my key (and kp + 8) in the first product
        const int v0 = key_of(2 * t4), v1 = key_of(2 * t4 + 1);   // my keys (and + 8) in the second
        uint32_t n = 0, nq = 0;
        const bool by_pair = join_by_pair(a.H_kv, pg.n_seq, a.n_slots);
        bool owner = false, ok = true;   // !ok: a wait gave up; the warp only keeps up with the others' barriers
        if (a.stall_ns != 0 && warp == 0) ok = warp_wait(&ms->stall, 0, s_abort, a.stall_ns);
        Piece p;
        // sequences without keys have no unit in the list
        for (int i = blockIdx.x; i < pg.n_seq; i += gridDim.x) {
            if (keys_of(pg, i) > 0) continue;
            for (int e = threadIdx.x; e < a.H_q * D; e += 32 * CW) store_out<DT>(a.out, (int64_t)i * a.H_q * D + e, 0.f);
            if (a.lse)
                for (int e = threadIdx.x; e < a.H_q; e += 32 * CW) a.lse[(int64_t)i * a.H_q + e] = -INFINITY;
            if (by_pair)
                for (int e = threadIdx.x; e < a.H_kv; e += 32 * CW) a.desc[e * pg.n_seq + i] = make_int4(0, 0, 0, 0);
        }
        while (walk.next(pg, a.H_kv, p)) {
            // the group's queries as the second operand of S^T: lane (g, t4) holds head g's eight values from
            // dimension 32 i + 8 t4 (q8_0, i a block) or 64 (i / 2) + 8 (t4 + 4 (i % 2)) (f16), for two steps each
            const int qs = nq % a.n_q;
            const uint32_t q_at = smem_u32(sm + C::OFF_Q) + qs * a.G * D * C::ESZ;
            ok = ok && warp_wait(&ms->q_full[qs], (nq / a.n_q) & 1, s_abort);
            uint32_t qf[D / 16][NT][2];
            [[maybe_unused]] float c0[C::NB][NT][2], worth[NT][2];
            if constexpr (Q4) {
                q4_queries<D, DT, NT>(q_at, a.G, a.scale_log2, lane, qf, c0, worth);
            } else {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int dim = Q8 || Q4 ? 32 * i + 8 * t4 : 64 * (i >> 1) + 8 * (t4 + 4 * (i & 1));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int head = nt * 8 + g;
                        uint32_t w[4] = {0u, 0u, 0u, 0u};
                        if (head < a.G) {
                            const uint32_t at = q_at + (head * D + dim) * C::ESZ;
                            const uint4 x = lds128(at);
                            const uint32_t xi[4] = {x.x, x.y, x.z, x.w};
                            if constexpr (DT == KVC_IN_F16) {
                                for (int e = 0; e < 4; ++e) w[e] = xi[e];
                            } else if constexpr (DT == KVC_IN_BF16) {
                                for (int e = 0; e < 4; ++e)
                                    w[e] = pack_half2(__uint_as_float(xi[e] << 16), __uint_as_float(xi[e] & 0xFFFF0000u));
                            } else {
                                const uint4 y = lds128(at + 16);
                                w[0] = pack_half2(__uint_as_float(x.x), __uint_as_float(x.y));
                                w[1] = pack_half2(__uint_as_float(x.z), __uint_as_float(x.w));
                                w[2] = pack_half2(__uint_as_float(y.x), __uint_as_float(y.y));
                                w[3] = pack_half2(__uint_as_float(y.z), __uint_as_float(y.w));
                            }
                        }
                        qf[2 * i][nt][0] = w[0]; qf[2 * i][nt][1] = w[1];
                        qf[2 * i + 1][nt][0] = w[2]; qf[2 * i + 1][nt][1] = w[3];
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms->q_empty[qs]);
            ++nq;

            float o[C::MT][NT][4], m[NT][2], l[NT][2];
            [[maybe_unused]] float ob[Q4 ? C::NB : 1][NT][4];
            [[maybe_unused]] __half2 d_most = __float2half2_rn(0.f);   // q4_0: the greatest scale of V so far
            [[maybe_unused]] float d_log2 = 0.f;                       // 2^d_log2 is above it
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt][0] = m[nt][1] = -INFINITY;
                l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                for (int i = 0; i < C::MT; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
                if constexpr (Q4)
#pragma unroll
                    for (int b = 0; b < C::NB; ++b) ob[b][nt][0] = ob[b][nt][1] = ob[b][nt][2] = ob[b][nt][3] = 0.f;
            }
            for (int t = p.t0; t < p.t1; ++t, ++n) {
                const int st = n % C::NS;
                ok = ok && warp_wait(&ms->full[st], (n / C::NS) & 1, s_abort);
                if (!ok) break;
                if constexpr (Q4) {
                    q4_tile<D, NT, C>(smem_u32(sm + st * C::STAGE), ms->count[st] + SUBS * warp, warp, lane, qf, c0, worth, o,
                                      ob, m, l, d_most, d_log2);
                } else if (const int count = ms->count[st][warp]; count > 0) {
                    const uint32_t kt = smem_u32(sm + st * C::STAGE), vt = kt + C::TILE, sc = vt + C::TILE;
                    const int ra = warp * 16 + kp, rb = ra + 8;   // my rows of the tile
                    float s[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
                    if constexpr (Q8) {
                        uint32_t da[C::NB / 2], db[C::NB / 2];   // scales of my two keys
                        if constexpr (D == 128) {
                            const uint2 x = lds64(sc + ra * 8), y = lds64(sc + rb * 8);
                            da[0] = x.x; da[1] = x.y; db[0] = y.x; db[1] = y.y;
                        } else {
                            da[0] = lds32(sc + ra * 4); db[0] = lds32(sc + rb * 4);
                        }
#pragma unroll
                        for (int b = 0; b < C::NB; ++b) {
                            const int c = 2 * b + (t4 >> 1);
                            const int sw = D == 128 ? c ^ (kp & 7) : c ^ ((kp >> 1) & 3);
                            const uint2 x = lds64(kt + ra * C::ROW + (sw << 4) + 8 * (t4 & 1));
                            const uint2 y = lds64(kt + rb * C::ROW + (sw << 4) + 8 * (t4 & 1));
                            float acc[NT][4];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t u = (j ? x.y : x.x) ^ 0x80808080u, w = (j ? y.y : y.x) ^ 0x80808080u;
                                const uint32_t A[4] = {unbias(__byte_perm(u, 0x64646464u, 0x4140)),
                                                       unbias(__byte_perm(w, 0x64646464u, 0x4140)),
                                                       unbias(__byte_perm(u, 0x64646464u, 0x4342)),
                                                       unbias(__byte_perm(w, 0x64646464u, 0x4342))};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_16816(acc[nt], A, qf[2 * b + j][nt][0], qf[2 * b + j][nt][1]);
                            }
                            const float2 fa = __half22float2(as_half2(da[b >> 1])), fb = __half22float2(as_half2(db[b >> 1]));
                            const float ca = b & 1 ? fa.y : fa.x, cb = b & 1 ? fb.y : fb.x;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                s[nt][0] = fmaf(acc[nt][0], ca, s[nt][0]);
                                s[nt][1] = fmaf(acc[nt][1], ca, s[nt][1]);
                                s[nt][2] = fmaf(acc[nt][2], cb, s[nt][2]);
                                s[nt][3] = fmaf(acc[nt][3], cb, s[nt][3]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            const uint32_t base = kt + (i >> 1) * KT * 128 + (((t4 + 4 * (i & 1)) ^ (kp & 7)) << 4);
                            const uint4 x = lds128(base + ra * 128), y = lds128(base + rb * 128);
                            const uint32_t A[4] = {x.x, y.x, x.y, y.y}, B[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma_16816(s[nt], A, qf[2 * i][nt][0], qf[2 * i][nt][1]);
                                mma_16816(s[nt], B, qf[2 * i + 1][nt][0], qf[2 * i + 1][nt][1]);
                            }
                        }
                    }
                    if (count < 16) {   // the last subtile of a sequence
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (kp >= count) s[nt][0] = s[nt][1] = -INFINITY;
                            if (kp + 8 >= count) s[nt][2] = s[nt][3] = -INFINITY;
                        }
                    }
                    bool above = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            above |= fmaxf(s[nt][e], s[nt][e + 2]) * a.scale_log2 > m[nt][e] + RESCALE_LOG2;
                    if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float f[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x = fmaxf(s[nt][e], s[nt][e + 2]);
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                                const float m_new = fmaxf(m[nt][e], x * a.scale_log2 - SHIFT_LOG2);
                                f[e] = m[nt][e] == m_new ? 1.f : ex2(m[nt][e] - m_new);
                                m[nt][e] = m_new;
                                l[nt][e] *= f[e];
                            }
#pragma unroll
                            for (int i = 0; i < C::MT; ++i) {
                                o[i][nt][0] *= f[0]; o[i][nt][1] *= f[1]; o[i][nt][2] *= f[0]; o[i][nt][3] *= f[1];
                            }
                        }
                    }
                    uint32_t pb[NT][2], pl[NT][2];   // the numerators in fp16, and what that leaves of them
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float e[4];
                        // a reference of -infinity (no score above it yet): the numerators are zero, or NaN where a score is
                        const float ref[2] = {m[nt][0] == -INFINITY ? 0.f : m[nt][0], m[nt][1] == -INFINITY ? 0.f : m[nt][1]};
#pragma unroll
                        for (int i = 0; i < 4; ++i) e[i] = ex2(fmaf(s[nt][i], a.scale_log2, -ref[i & 1]));
                        l[nt][0] += e[0] + e[2];
                        l[nt][1] += e[1] + e[3];
                        const uint32_t p0 = pack_half2(e[0], e[1]), p1 = pack_half2(e[2], e[3]);
                        pb[nt][0] = movmatrix_trans(p0);
                        pb[nt][1] = movmatrix_trans(p1);
                        if constexpr (C::FINE) {
                            const float2 f0 = __half22float2(as_half2(p0)), f1 = __half22float2(as_half2(p1));
                            pl[nt][0] = movmatrix_trans(pack_half2(e[0] - f0.x, e[1] - f0.y));
                            pl[nt][1] = movmatrix_trans(pack_half2(e[2] - f1.x, e[3] - f1.y));
                        }
                    }
                    if constexpr (Q8) {
                        constexpr int NW = D / 32;   // words of one key's part: 16 (8) dimensions from D / 8 * g
                        uint32_t w[4][NW], d[4];
                        const int keys[4] = {v0, v1, v0 + 8, v1 + 8};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = warp * 16 + keys[i];
                            if constexpr (D == 128) {
                                const uint4 x = lds128(vt + key * 128 + ((g ^ (keys[i] & 7)) << 4));
                                w[i][0] = x.x; w[i][1] = x.y; w[i][2] = x.z; w[i][3] = x.w;
                            } else {
                                const uint2 x = lds64(vt + key * 64 + (((g >> 1) ^ ((keys[i] >> 1) & 3)) << 4) + 8 * (g & 1));
                                w[i][0] = x.x; w[i][1] = x.y;
                            }
                            d[i] = lds16(sc + C::SC + (key * C::NB + (g * (D / 8)) / 32) * 2);
                        }
                        const __half2 d01 = as_half2(d[0] | d[1] << 16), d23 = as_half2(d[2] | d[3] << 16);
#pragma unroll
                        for (int i = 0; i < C::MT; ++i) {
                            uint32_t A[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {   // row half e & 1 (the odd byte), keys 2 (e / 2) and + 1
                                const int b = 2 * (i & 1) + (e & 1);
                                uint32_t u = __byte_perm(w[e & 2][i >> 1], w[(e & 2) + 1][i >> 1], 0x11u * b | 0x1100u * (4 + b));
                                u = (u & 0x00FF00FFu) ^ 0x64806480u;
                                A[e] = as_u32(__hmul2(as_half2(unbias(u)), e & 2 ? d23 : d01));
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma_16816(o[i][nt], A, pb[nt][0], pb[nt][1]);
                                if constexpr (C::FINE) mma_16816(o[i][nt], A, pl[nt][0], pl[nt][1]);
                            }
                        }
                    } else {
                        const int key = warp * 16 + key_of(lane & 7) + 8 * (lane >> 4);
#pragma unroll
                        for (int i = 0; i < C::MT; ++i) {
                            const int c = 2 * i + ((lane >> 3) & 1);
                            uint32_t A[4];
                            ldmatrix_x4_trans(A, vt + (c >> 3) * KT * 128 + key * 128 + (((c & 7) ^ (key & 7)) << 4));
                            if (count < 16) {   // values behind the sequence may be anything: their weight is zero
                                const uint32_t lo = (v0 < count ? 0xFFFFu : 0u) | (v1 < count ? 0xFFFF0000u : 0u);
                                const uint32_t hi = (v0 + 8 < count ? 0xFFFFu : 0u) | (v1 + 8 < count ? 0xFFFF0000u : 0u);
                                A[0] &= lo; A[1] &= lo; A[2] &= hi; A[3] &= hi;
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_16816(o[i][nt], A, pb[nt][0], pb[nt][1]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms->empty[st]);
            }

            if constexpr (Q4) {
                // the nibbles' places in their words (rows 0 to 7 of a tile: the lower), and the 8 that is in each of them
#pragma unroll
                for (int i = 0; i < C::MT; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[i][nt][e] = fmaf(o[i][nt][e], e < 2 ? 0x1p24f : 0x1p20f, -0x1p20f * ob[i >> 1][nt][e]);
            }
            // ---- the piece is done: join the four warps.  Warp w ends up with tiles [w OWN, (w + 1) OWN) of O^T.
            float f[NT][2], M[NT][2], L[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[nt][e];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    l[nt][e] = x;
                    if (g == 0) ms->ml[warp][nt * 8 + 2 * t4 + e] = make_float2(m[nt][e], x);
                }
            named_barrier(1, 32 * CW);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int head = nt * 8 + 2 * t4 + e;
                    float2 x[CW];
                    float mx = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int w = 0; w < CW; ++w) {
                        x[w] = ms->ml[w][head];
                        mx = fmaxf(mx, x[w].x);
                    }
#pragma unroll
                    for (int w = 0; w < CW; ++w) sum += x[w].x == -INFINITY ? x[w].y : x[w].y * ex2(x[w].x - mx);   // zero or NaN
                    M[nt][e] = mx;
                    L[nt][e] = sum;
                    f[nt][e] = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - mx);
                }
            float4 *red = reinterpret_cast<float4 *>(sm + C::OFF_RED);
#pragma unroll
            for (int i = 0; i < C::MT; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    o[i][nt][0] *= f[nt][0]; o[i][nt][1] *= f[nt][1]; o[i][nt][2] *= f[nt][0]; o[i][nt][3] *= f[nt][1];
                    const int to = i / C::OWN;
                    if (to != warp)
                        red[((i * NT + nt) * (CW - 1) + ((warp - to - 1) & 3)) * 32 + lane] =
                            make_float4(o[i][nt][0], o[i][nt][1], o[i][nt][2], o[i][nt][3]);
                }
            named_barrier(1, 32 * CW);
            const bool whole = p.t0 == 0 && p.t1 == p.nt;
            const int slot = (blockIdx.x * 2 + (p.t0 == 0)) * a.G;
#pragma unroll
            for (int i = 0; i < C::MT; ++i) {
                if (i / C::OWN != warp) continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int x = 0; x < CW - 1; ++x) {
                        const float4 y = red[((i * NT + nt) * (CW - 1) + x) * 32 + lane];
                        o[i][nt][0] += y.x; o[i][nt][1] += y.y; o[i][nt][2] += y.z; o[i][nt][3] += y.w;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int head = nt * 8 + 2 * t4 + (e & 1);
                        const int dim = Q4 ? 32 * (i >> 1) + 8 * (g >> 1) + (g & 1) + 4 * (i & 1) + 2 * (e >> 1)
                                      : Q8 ? g * (D / 8) + 2 * i + (e >> 1) : 16 * i + g + 8 * (e >> 1);
                        if (head >= a.G) continue;
                        if (whole)
                            store_out<DT>(a.out, ((int64_t)p.seq * a.H_q + p.h * a.G + head) * D + dim,
                                          L[nt][e & 1] > 0.f || L[nt][e & 1] != L[nt][e & 1] ? o[i][nt][e] / L[nt][e & 1] : 0.f);
                        else
                            a.part_o[(int64_t)(slot + head) * D + dim] = o[i][nt][e];
                    }
                }
            }
            if (warp == 0 && g == 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int head = nt * 8 + 2 * t4 + e;
                        if (head >= a.G) continue;
                        if (!whole)   // the join passes over parts with M = -infinity, but a NaN has to reach it
                            a.part_ml[slot + head] = make_float2(isnan(L[nt][e]) ? INFINITY : M[nt][e], L[nt][e]);
                        else if (a.lse)
                            a.lse[(int64_t)p.seq * a.H_q + p.h * a.G + head] =
                                L[nt][e] == 0.f ? -INFINITY : (M[nt][e] + log2f(L[nt][e])) * LN2;
                    }
            }
            if (p.t0 == 0 && (by_pair || !whole)) {
                owner = true;
                if (threadIdx.x == 0) {
                    const unsigned long long end = u1 + (p.nt - p.t1);   // the pair's last unit, plus one
                    const int last = (int)((end * runs_of(W) - 1) / W);    // the CTA whose run holds it
                    a.desc[by_pair ? p.h * pg.n_seq + p.seq : blockIdx.x] =
                        make_int4(p.seq, p.h, whole ? 0 : last - (int)blockIdx.x + 1, blockIdx.x);
                }
            }
        }
        if (!by_pair && !owner && threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    if (*s_abort) {   // a wait gave up, whoever's: let the copies in flight land before the CTA exits
        if (threadIdx.x == 0) atomicExch(&g_paged_status, 1);
        if (warp == CW) {
            volatile int never = 0;
            const uint32_t n = ms->tiles, nq = ms->queries, n_q = a.n_q;
            for (uint32_t e = n > (uint32_t)C::NS ? n - C::NS : 0; e < n; ++e)
                mbar_wait(&ms->full[e % C::NS], (e / C::NS) & 1, &never, 200000000ull);
            for (uint32_t e = nq > n_q ? nq - n_q : 0; e < nq; ++e)
                mbar_wait(&ms->q_full[e % n_q], (e / n_q) & 1, &never, 200000000ull);
        }
    }
}

// Joins the partials of one pair: for each query head
// out = sum_p w_p O_p / sum_p w_p l_p, w_p = 2^(m_p - max m), the runs in a fixed order.  D / 4 threads, a group, take a
// row.  Where there are few pairs a CTA joins one head (blockIdx.y), its groups sharing the partials; else (MANY) a CTA
// joins all heads, a group each where there are few partials: 96 sequences of 64 tokens take 12.2 us, 13.5 with a CTA for
// each head, which is mostly the starting of CTAs.  The 96 sequences of 5 to 16,384 with a group for a head up to 0, 2, 8 and 32
// partials: 82, 82, 79 and 79 us, in 16 heads to a group 136, 135, 125 and 125.
constexpr int FEW_PARTS = 8;
template <int D, int DT, bool MANY>
__global__ void __launch_bounds__(COMBINE_THREADS) combine_paged_kernel(const Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int4 d = __ldcg(a.desc + blockIdx.x);
    if (d.z == 0) return;
    constexpr int LANES = D / 4, GROUPS = COMBINE_THREADS / LANES;
    const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    // partials first, first + step, ... of a head
    auto join = [&](int head, int first, int step, float &m, float &l, float4 &acc) {
        m = -INFINITY;
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // partial j lies with CTA d.w + j: its second slot for the first (the pair begins there), else the first
        constexpr int B = 4;
        for (int j0 = first; j0 < d.z; j0 += B * step) {
            float2 ml[B];
            float4 o[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int j = j0 + b * step;
                ml[b] = make_float2(-INFINITY, 0.f);
                o[b] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < d.z) {
                    const int slot = ((d.w + j) * 2 + (j == 0)) * a.G + head;
                    ml[b] = __ldcg(a.part_ml + slot);
                    o[b] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + (int64_t)slot * D) + lane);
                }
            }
            float mx = m;
#pragma unroll
            for (int b = 0; b < B; ++b) mx = fmaxf(mx, ml[b].x);
            if (mx == -INFINITY) continue;
            const float f = m == -INFINITY ? 0.f : ex2(m - mx);
            m = mx;
            l *= f; acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const float w = ml[b].x == -INFINITY ? 0.f : ex2(ml[b].x - m);
                l = fmaf(w, ml[b].y, l);
                acc.x = fmaf(w, o[b].x, acc.x); acc.y = fmaf(w, o[b].y, acc.y);
                acc.z = fmaf(w, o[b].z, acc.z); acc.w = fmaf(w, o[b].w, acc.w);
            }
        }
    };
    auto store = [&](int head, float M, float L, const float4 &acc) {
        const int64_t row = (int64_t)d.x * a.H_q + d.y * a.G + head;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        store_out<DT>(a.out, row * D + 4 * lane, acc.x * inv);
        store_out<DT>(a.out, row * D + 4 * lane + 1, acc.y * inv);
        store_out<DT>(a.out, row * D + 4 * lane + 2, acc.z * inv);
        store_out<DT>(a.out, row * D + 4 * lane + 3, acc.w * inv);
        if (a.lse && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
    };
    float m, l;
    float4 acc;
    if (MANY && d.z <= FEW_PARTS) {
        for (int head = grp; head < a.G; head += GROUPS) {
            join(head, 0, 1, m, l, acc);
            store(head, m, l, acc);
        }
        return;
    }
    __shared__ float sm_m[GROUPS], sm_l[GROUPS];
    __shared__ float4 sm_o[GROUPS][LANES];
    for (int head = MANY ? 0 : blockIdx.y, end = MANY ? a.G : head + 1; head < end; ++head) {
        join(head, grp, GROUPS, m, l, acc);
        if (MANY) __syncthreads();   // the groups' results of the head before have been read
        if (lane == 0) { sm_m[grp] = m; sm_l[grp] = l; }
        sm_o[grp][lane] = acc;
        __syncthreads();
        if (grp != 0) continue;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) M = fmaxf(M, sm_m[i]);
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const float w = sm_m[i] == -INFINITY ? 0.f : ex2(sm_m[i] - M);
            const float4 o = sm_o[i][lane];
            L = fmaf(w, sm_l[i], L);
            acc.x = fmaf(w, o.x, acc.x); acc.y = fmaf(w, o.y, acc.y);
            acc.z = fmaf(w, o.z, acc.z); acc.w = fmaf(w, o.w, acc.w);
        }
        store(head, M, L, acc);
    }
}

template <int D, int CT, int DT, int NT>
int launch_t(const CUtensorMap &tk, const CUtensorMap &tv, const PagedView &pg, Args a, cudaStream_t s) {
    using C = Cfg<D, CT, DT, NT>;
    a.n_q = min(MAX_NQ, C::Q_ROOM / (a.G * D * C::ESZ));
    if (allow_dynamic_smem((const void *)decode_paged_kernel<D, CT, DT, NT>, smem_budget(CT, NT)) != KVC_OK) return KVC_ECUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.n_slots);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_budget(CT, NT);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, decode_paged_kernel<D, CT, DT, NT>, tk, tv, pg, a) != cudaSuccess) return KVC_ECUDA;
    const bool by_pair = join_by_pair(a.H_kv, pg.n_seq, a.n_slots);
    cfg.gridDim = by_pair ? dim3(a.H_kv * pg.n_seq, a.G) : dim3(a.n_slots);
    cfg.blockDim = dim3(COMBINE_THREADS);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, by_pair ? combine_paged_kernel<D, DT, false> : combine_paged_kernel<D, DT, true>, a) != cudaSuccess)
        return KVC_ECUDA;
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ECUDA;
}

template <int D, int CT>
int launch_d(int dtype, const CUtensorMap &tk, const CUtensorMap &tv, const PagedView &pg, const Args &a, cudaStream_t s) {
    switch (dtype) {
#define KVC_CASE(DT)                                                                             \
    case DT:                                                                                     \
        return a.G <= 8 ? launch_t<D, CT, DT, 1>(tk, tv, pg, a, s) : launch_t<D, CT, DT, 2>(tk, tv, pg, a, s);
        KVC_CASE(KVC_IN_F32)
        KVC_CASE(KVC_IN_BF16)
        KVC_CASE(KVC_IN_F16)
#undef KVC_CASE
        default: return KVC_EINVAL;
    }
}

// The tensor maps of a layer and the launch; Args as decode_paged.cu fills them.
template <int CT>
int launch_type(const kvc_cache &c, int layer, int page_size, int dtype, const PagedView &pg, Args a, cudaStream_t s) {
    const kvc_desc &d = c.d;
    const Geom g = geom_of(d);
    const int D = d.head_dim;
    // a TMA box covers the part of a tile that lies in one page
    constexpr int KT = keys_per_tile(CT);
    a.box = 16;
    while (a.box < KT && page_size % (2 * a.box) == 0) a.box *= 2;
    const CUtensorMapDataType dt = CT == KVC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapSwizzle sw = CT == KVC_Q4_0 ? D == 64 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B
                                  : CT == KVC_Q8_0 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    const uint32_t row = CT == KVC_Q4_0 ? D / 2 : D, inner = CT == KVC_F16 ? 64 : row;   // elements of the map
    CUtensorMap tk, tv;
    auto map = [&](CUtensorMap *m, const void *base) {
        return make_map_3d(m, dt, static_cast<const uint8_t *>(base) + code_bytes(CT, layer * g.c_layer), row, d.n_ctx,
                           d.n_head_kv, code_bytes(CT, g.c_tok), code_bytes(CT, g.c_head), inner, a.box, 1, sw);
    };
    if (!map(&tk, c.k_q) || !map(&tv, c.v_q)) return KVC_ECUDA;
    return D == 128 ? launch_d<128, CT>(dtype, tk, tv, pg, a, s) : launch_d<64, CT>(dtype, tk, tv, pg, a, s);
}

int read_and_clear(int32_t *status) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(int)) != cudaSuccess) return KVC_ECUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int)) != cudaSuccess) return KVC_ECUDA;
    *status = v;
    return KVC_OK;
}

}  // namespace
}  // namespace kvc
