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
#include "decode_paged.cuh"

namespace kvc {

// set by a kernel of this file that gave up a bounded wait (read and cleared with the other kernels' status)
__device__ int g_paged_status;

namespace {

using namespace paged;

constexpr int KT = 64;              // keys per tile
constexpr int CW = 4;               // consumer warps, 16 keys of a tile each
constexpr int THREADS = 32 * (CW + 1);
// CTAs per SM: two, whose consumers keep up with the loads of an f16 pool; three for q8_0, where they do not, but for groups
// of more than 8 query heads (NT = 2), whose accumulators three leave too few registers.  With three and two, in us (bf16, 8
// kv heads, back to back): up to 8 heads to a group, D = 128 the 96 sequences below 79 and 83, one of 58,300 31.7 and 32.2, 96
// of 700 40.9 and 38.1; D = 64 68 and 69, 21.6 and 25.5.  16 heads, D = 128 144 and 125, 50 and 43; D = 64 70 and 73: there
// two are 5% slower.
constexpr int ctas_per_sm(bool q8, int NT) { return q8 && NT == 1 ? 3 : 2; }
constexpr int smem_budget(bool q8, int NT) { return ctas_per_sm(q8, NT) == 3 ? 76800 : 115712; }   // 75 and 113 KB
constexpr int MAX_NS = 10;          // tiles of the longest ring (16 heads of 64, q8_0)
// What starting and ending a pair costs, in tiles.  With 0, 1, 2 and 4, in us (q8_0, bf16): 96 sequences of 5 to 16,384 91, 85,
// 79 and 87, in 16 heads to a group 136, 131, 125 and 112, with D = 64 61, 57, 68 and 72, f16 123, 119, 120 and 120; 170 sequences
// of 10 to 3,000, 2 kv heads 25, 20, 19 and 21; one of 58,300 31.4, 31.4, 31.7 and 31.6.  (The cuts' places, and with them
// which CTAs pass the same tokens together, move with it.)
constexpr int PIECE_COST = 2;
template <int D, bool Q8, int DT, int NT>
struct Cfg {
    // Both operands of a q8_0 pool's second product are rounded to fp16, which an fp16 or float32 output shows (the 96
    // sequences above: 1.53 times the error of the output's own rounding): there the numerators enter in two parts, for 4%
    // of the time (1.41 times).  A bf16 output's rounding, eight times as coarse, hides it.
    static constexpr bool FINE = Q8 && DT != KVC_IN_BF16;
    static constexpr int NB = D / 32;                       // q8_0 blocks per row
    static constexpr int ROW = D * (Q8 ? 1 : 2);            // bytes of a row
    static constexpr int TILE = KT * ROW;                   // a K or V tile
    static constexpr int SC = Q8 ? KT * NB * 2 : 0;         // a tile's scales
    static constexpr int STAGE = 2 * TILE + ((2 * SC + 1023) & ~1023);
    static constexpr int MT = D / 16;                       // 16-row tiles of O^T
    static constexpr int OWN = MT / CW;                     // of which each warp writes
    static constexpr int RED = MT * NT * (CW - 1) * 512;    // the other warps' accumulators
    static constexpr int ESZ = DT == KVC_IN_F32 ? 4 : 2;
    static constexpr int QB = 8 * NT * D * ESZ;             // the most that a group's queries take
    static constexpr int MISC = 1024;
    static constexpr int FIT = (smem_budget(Q8, NT) - 1024 - RED - QB - MISC) / STAGE;
    static constexpr int NS = FIT < MAX_NS ? FIT : MAX_NS;
    static constexpr int OFF_RED = NS * STAGE, OFF_MISC = OFF_RED + RED, OFF_Q = OFF_MISC + MISC;
    static constexpr int Q_ROOM = smem_budget(Q8, NT) - 1024 - OFF_Q;
    static_assert(NS >= 2 && Q_ROOM >= QB, "shared memory plan");
};
constexpr int MAX_NQ = 4;           // slots for the queries of pieces to come: as many as fit (1, 2 and 4 take the same time)

// what the small area behind the ring holds
struct Misc {
    uint64_t full[MAX_NS], empty[MAX_NS], q_full[MAX_NQ], q_empty[MAX_NQ], stall;
    int count[MAX_NS][CW];               // keys of each subtile that exist
    float2 ml[CW][16];                   // reference and sum of each warp and head
    unsigned long long warp_units[CW + 1], total;
    uint32_t tiles, queries;             // what the producer has asked for in all
    int first_seq, rest, abort;
};
static_assert(sizeof(Misc) <= 1024, "small area");

// the order of the eight keys of half a subtile: rows 2i and 2i+1 differ in bit 2, even rows (and odd rows) in bits
// 1 and 2, which is what makes every swizzled read below free of bank conflicts (a row of 128 bytes)
__device__ __forceinline__ int key_of(int r) { return r ^ ((r & 1) << 2); }

// bytes c ^ 0x80 under the high byte 0x64 are the fp16 numbers 1152 + c
__device__ __forceinline__ uint32_t unbias(uint32_t u) { return as_u32(__hsub2(as_half2(u), as_half2(0x64806480u))); }
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}

template <int D, bool Q8, int DT, int NT>
__global__ void __launch_bounds__(THREADS, ctas_per_sm(Q8, NT))
    decode_paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const PagedView pg, const Args a) {
    using C = Cfg<D, Q8, DT, NT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    Misc *ms = reinterpret_cast<Misc *>(sm + C::OFF_MISC);
    volatile int *s_abort = &ms->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ms->abort = 0;
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&ms->full[s], Q8 ? 33 : 1);
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
        for (int i = i0; i < i1; ++i) mine += units_of<KT, PIECE_COST>(keys_of(pg, i));
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
        unsigned long long r = total ? run_start(total * a.H_kv, gridDim.x, blockIdx.x) % total : 0;
        if (threadIdx.x == 0) ms->total = total;
        if (r >= before && r < before + mine) {
            r -= before;
            int i = i0;
            for (; i + 1 < i1; ++i) {
                const unsigned long long n = units_of<KT, PIECE_COST>(keys_of(pg, i));
                if (r < n) break;
                r -= n;
            }
            ms->first_seq = i;
            ms->rest = (int)r;
        }
        __syncthreads();
    }
    const unsigned long long W = ms->total * a.H_kv, u0 = run_start(W, gridDim.x, blockIdx.x), u1 = run_start(W, gridDim.x, blockIdx.x + 1);
    Walk<KT, PIECE_COST> walk(pg, u1 > u0 ? ms->first_seq : 0, u1 > u0 ? (int)(u0 / ms->total) : 0, u1 > u0 ? ms->rest : 0, u1 - u0);

    if (warp == CW) {
        // ------------------------------------------------------------------ producer
        // Tiles are taken eight at a time, across pieces: lane 4 i + j knows subtile j of the i-th.  The pages of the
        // next eight are being looked up while these are copied.
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
            while (b.n < 8 && more) {
                const bool first = t >= p.t1;
                if (first) {
                    more = walk.next(pg, a.H_kv, p);
                    if (!more) break;
                    t = p.t0;
                }
                if ((lane >> 2) == b.n) {
                    b.seq = p.seq; b.h = p.h; b.t = t; b.keys = p.keys; b.first = first;
                }
                ++t;
                ++b.n;
            }
            const int key = b.t * KT + (lane & 3) * 16;
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
            const int key0 = cur.t * KT + (lane & 3) * 16;
            // my subtile's first pool position (-1: none of its keys exist) and how many of its keys exist
            const int slot = (unsigned)cur.page < (unsigned)pg.n_pages ? cur.page * pg.page_size + key0 % pg.page_size : -1;
            const int count = slot < 0 ? 0 : min(16, cur.keys - key0);
            for (int i = 0; i < cur.n; ++i) {
                const int h = __shfl_sync(0xffffffffu, cur.h, 4 * i);
                if (__shfl_sync(0xffffffffu, (int)cur.first, 4 * i)) {
                    const int qs = nq % a.n_q, seq = __shfl_sync(0xffffffffu, cur.seq, 4 * i);
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
                if ((lane >> 2) == i) ms->count[st][lane & 3] = count;
                const int box_slot = __shfl_sync(0xffffffffu, slot, 4 * i + ((lane * per_box) & 3));
                const bool load = lane < boxes && box_slot >= 0;
                const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
                __syncwarp();   // the counts before the arrival that publishes them (shuffles and ballots order no memory)
                if (lane == 0) mbar_arrive_expect_tx(&ms->full[st], loads * 2 * a.box * C::ROW);
                __syncwarp();
                if (load) {
                    const int off = lane * a.box * (Q8 ? C::ROW : 128);
#pragma unroll
                    for (int hh = 0; hh < (Q8 ? 1 : D / 64); ++hh) {
                        tma_load_3d(kt + hh * KT * 128 + off, &tm_k, &ms->full[st], hh * 64, box_slot, h);
                        tma_load_3d(vt + hh * KT * 128 + off, &tm_v, &ms->full[st], hh * 64, box_slot, h);
                    }
                }
                if constexpr (Q8) {
                    uint8_t *sc = vt + C::TILE;
#pragma unroll
                    for (int x = 0; x < 2 * KT / 32; ++x) {
                        const int key = (x * 32 + lane) & (KT - 1), is_v = x / (KT / 32);
                        const int sl = __shfl_sync(0xffffffffu, slot, 4 * i + (key >> 4));
                        const bool valid = (key & 15) < __shfl_sync(0xffffffffu, count, 4 * i + (key >> 4));
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
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int dim = Q8 ? 32 * i + 8 * t4 : 64 * (i >> 1) + 8 * (t4 + 4 * (i & 1));
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms->q_empty[qs]);
            ++nq;

            float o[C::MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt][0] = m[nt][1] = -INFINITY;
                l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                for (int i = 0; i < C::MT; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
            }
            for (int t = p.t0; t < p.t1; ++t, ++n) {
                const int st = n % C::NS;
                ok = ok && warp_wait(&ms->full[st], (n / C::NS) & 1, s_abort);
                if (!ok) break;
                const int count = ms->count[st][warp];
                if (count > 0) {
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
                    // In powers of two, and rounded before the reference is taken off, as the reference was: fused, the greatest score
                    // less its reference would be off by the reference's rounding, which passes any exponent where scores pass 2^27.
                    const uint64_t scale2 = f2_pack(a.scale_log2, a.scale_log2);
                    bool above = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        f2_unpack(f2_mul(f2_pack(s[nt][0], s[nt][1]), scale2), s[nt][0], s[nt][1]);
                        f2_unpack(f2_mul(f2_pack(s[nt][2], s[nt][3]), scale2), s[nt][2], s[nt][3]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) above |= fmaxf(s[nt][e], s[nt][e + 2]) > m[nt][e] + RESCALE_LOG2;
                    }
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
                                const float m_new = fmaxf(m[nt][e], x - SHIFT_LOG2);
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
                        for (int i = 0; i < 4; i += 2) {
                            f2_unpack(f2_add(f2_pack(s[nt][i], s[nt][i + 1]), f2_pack(-ref[0], -ref[1])), e[i], e[i + 1]);
                            e[i] = ex2(e[i]);
                            e[i + 1] = ex2(e[i + 1]);
                        }
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
                        const int dim = Q8 ? g * (D / 8) + 2 * i + (e >> 1) : 16 * i + g + 8 * (e >> 1);
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
                    const int last = (int)((end * runs_of(W, gridDim.x) - 1) / W);    // the CTA whose run holds it
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

template <int D, bool Q8, int DT, int NT>
int launch_t(const CUtensorMap &tk, const CUtensorMap &tv, const PagedView &pg, Args a, cudaStream_t s) {
    using C = Cfg<D, Q8, DT, NT>;
    a.n_q = min(MAX_NQ, C::Q_ROOM / (a.G * D * C::ESZ));
    if (allow_dynamic_smem((const void *)decode_paged_kernel<D, Q8, DT, NT>, smem_budget(Q8, NT)) != KVC_OK) return KVC_ECUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.n_slots);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_budget(Q8, NT);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, decode_paged_kernel<D, Q8, DT, NT>, tk, tv, pg, a) != cudaSuccess) return KVC_ECUDA;
    const bool by_pair = join_by_pair(a.H_kv, pg.n_seq, a.n_slots);
    cfg.gridDim = by_pair ? dim3(a.H_kv * pg.n_seq, a.G) : dim3(a.n_slots);
    cfg.blockDim = dim3(COMBINE_THREADS);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, by_pair ? combine_paged_kernel<D, DT, false> : combine_paged_kernel<D, DT, true>, a,
                           (int)cfg.gridDim.x) != cudaSuccess)
        return KVC_ECUDA;
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ECUDA;
}

template <int D, bool Q8>
int launch_d(int dtype, const CUtensorMap &tk, const CUtensorMap &tv, const PagedView &pg, const Args &a, cudaStream_t s) {
    switch (dtype) {
#define KVC_CASE(DT)                                                                             \
    case DT:                                                                                     \
        return a.G <= 8 ? launch_t<D, Q8, DT, 1>(tk, tv, pg, a, s) : launch_t<D, Q8, DT, 2>(tk, tv, pg, a, s);
        KVC_CASE(KVC_IN_F32)
        KVC_CASE(KVC_IN_BF16)
        KVC_CASE(KVC_IN_F16)
#undef KVC_CASE
        default: return KVC_EINVAL;
    }
}

int slots_of(bool q8, int G) { return ctas_per_sm(q8, G <= 8 ? 1 : 2) * sm_count(); }

}  // namespace

size_t paged_scratch_bytes(const kvc_desc &d, int, int n_head_q) {
    const size_t G = n_head_q / d.n_head_kv;
    const int n = d.type == KVC_Q4_0 ? paged_q4_slots((int)G) : slots_of(d.type == KVC_Q8_0, (int)G);
    return (size_t)n * (2 * G * (d.head_dim + 2) * sizeof(float) + sizeof(int4));
}

int launch_decode_paged(const kvc_cache &c, const kvc_pages &p, int layer, const void *q, int64_t ld_q, int dtype,
                        int n_head_q, void *out, float *lse, void *scratch, cudaStream_t s) {
    const kvc_desc &d = c.d;
    const Geom g = geom_of(d);
    const bool q8 = d.type == KVC_Q8_0, q4 = d.type == KVC_Q4_0;
    const int esz = q8 ? 1 : 2, D = d.head_dim;
    Args a;
    a.ks = q8 || q4 ? static_cast<const uint16_t *>(c.k_s) + layer * g.s_layer : nullptr;
    a.vs = q8 || q4 ? static_cast<const uint16_t *>(c.v_s) + layer * g.s_layer : nullptr;
    a.s_tok = g.s_tok;
    a.s_head = g.s_head;
    a.q = static_cast<const uint8_t *>(q);
    a.ld_q = ld_q * dtype_bytes(dtype);
    a.out = out;
    a.lse = lse;
    a.H_q = n_head_q;
    a.H_kv = d.n_head_kv;
    a.G = n_head_q / d.n_head_kv;
    a.n_slots = q4 ? paged_q4_slots(a.G) : slots_of(q8, a.G);
    a.step = 1;
    a.desc = static_cast<int4 *>(scratch);
    a.part_o = reinterpret_cast<float *>(a.desc + a.n_slots);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)a.n_slots * 2 * a.G * D);
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)D);
    if (q4) return launch_decode_paged_q4(c, p, layer, dtype, a, s);   // no wait of its kernel can be made to run out
    a.stall_ns = take_test_stall(KVC_TEST_PAGED);
    // a TMA box covers the part of a tile that lies in one page
    a.box = p.page_size % 64 == 0 ? 64 : p.page_size % 32 == 0 ? 32 : 16;
    const CUtensorMapDataType dt = q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle sw = q8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap tk, tv;
    const uint32_t inner = q8 ? D : 64;
    auto map = [&](CUtensorMap *m, const void *base) {
        return make_map_3d(m, dt, static_cast<const uint8_t *>(base) + layer * g.c_layer * esz, D, d.n_ctx, d.n_head_kv,
                           g.c_tok * esz, g.c_head * esz, inner, a.box, 1, sw);
    };
    if (!map(&tk, c.k_q) || !map(&tv, c.v_q)) return KVC_ECUDA;
    const PagedView pg = paged_view(c, p);
    if (D == 128) return q8 ? launch_d<128, true>(dtype, tk, tv, pg, a, s) : launch_d<128, false>(dtype, tk, tv, pg, a, s);
    return q8 ? launch_d<64, true>(dtype, tk, tv, pg, a, s) : launch_d<64, false>(dtype, tk, tv, pg, a, s);
}

int read_and_clear_paged_status(int32_t *status) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(int)) != cudaSuccess) return KVC_ECUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int)) != cudaSuccess) return KVC_ECUDA;
    *status = v;
    return KVC_OK;
}

}  // namespace kvc
