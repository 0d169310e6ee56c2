// Causal attention of packed prompts with grouped heads, on the fifth-generation tensor cores.
//
// Sequence s has nq query rows and nk keys; row i sees the keys j <= i + nk - nq:
//   out[i][h] = sum_j softmax_j(q[i][h] . k[j][h/G] / sqrt(D)) v[j][h/G].
// Both products are contractions of the inputs' own type (bf16 or fp16) with float32 accumulators in tensor
// memory; the softmax runs in one pass over the keys with the row's running maximum and sum in float32.  What
// bounds it is the tensor cores' rate for long prompts, and for short ones the chain load - product - softmax -
// product - store of each block.
//
// Work split.  The G query heads of a kv head see the same keys, so a tile of 128 rows holds 128 / G tokens
// with all their heads: a prompt of 25 tokens with five heads fills one tile where a tile for each head would
// leave four fifths of five empty.  A block is two such tiles of a (sequence, kv head), which share each K and V tile of 128 keys.  The
// blocks of all kv heads and sequences, each as long as the keys that it sees plus a charge, form one list that
// is cut into equal runs, one for each CTA (one per SM); lengths are read on the device.  A block cut by a run's
// end leaves partial results (O, maximum, sum; at most two blocks for each CTA) that a second kernel joins in the
// runs' order; cuts close to a block's end move there.
//
// Tensor memory (512 columns): for each of the two tiles S (128 columns, then overwritten by P as 16-bit
// pairs, the A operand of the second product) and O (D columns).  The MMA thread alternates between the tiles - PV(k)
// and QK(k+1) of one run while the other's softmax does - and the MMAs of one thread execute in order, so QK(k+1) may
// be issued as soon as PV(k) is, although it overwrites the P that PV(k) reads.
//
// One CTA (12 warps):
//   warp 0     producer: walks the CTA's run of the list, passes each block on through a ring of items and
//              loads Q tiles and a ring of K and V tiles (in the order K(0) V(0) K(1) V(1) ...) by TMA;
//   warp 1     allocates tensor memory; one lane issues the MMAs;
//   warps 4-7, 8-11   softmax of the first and the second tile, a thread for each row: the row's maximum needs no
//              exchange between threads.  A tile's QK - softmax - PV is a chain, so PV starts on the first 64 keys
//              while the numerators of the others are computed.  O is rescaled only when the running maximum has grown by
//              more than 2^8.  Where a sequence ends inside a V tile they also set the rows behind it to zero.
// Every mbarrier wait is bounded (2 s); a wait that gives up sets the device status word.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "ptx.cuh"

namespace kvc {

// set by a kernel of this file that gave up a bounded wait (read and cleared with the other kernels' status)
__device__ int g_packed_status;

namespace {

using namespace ptx;

constexpr int BM = 128;             // rows of a tile
constexpr int BN = 128;             // keys of a tile
constexpr int THREADS = 384;        // a warpgroup with the producer and the MMA warp, two of softmax
constexpr int NI = 4;               // items on their way from the producer
constexpr int BLOCK_COST = 128;     // what a block costs besides its keys, in keys
constexpr int SNAP = 2;             // a cut fewer tiles than this from an end of a block moves there
constexpr int MAX_DYN_SMEM = 232448;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr float LN2 = 0.69314718055994531f;
constexpr uint32_t TMEM_COLS = 512;

template <int D>
struct Cfg {
    static constexpr int TILE = 128 * D * 2;               // a Q, K or V tile
    static constexpr int NS = D == 128 ? 5 : 11;            // ring of K and V tiles
    static constexpr int OFF_Q = 0, OFF_RING = 2 * TILE, OFF_MISC = OFF_RING + NS * TILE;
    static constexpr int USED = OFF_MISC + 1024;
    static constexpr int ALLOC = USED + 1024 <= MAX_DYN_SMEM ? USED + 1024 : MAX_DYN_SMEM;
    static_assert(USED <= MAX_DYN_SMEM, "shared memory plan");
    static constexpr uint32_t COL_S = 0, COL_O = 256;       // tile x: S at 128 x, O at 256 + D x
};

// A block, or the part of its keys that falls into this CTA's run.
struct Item {
    int q_row, tokens;        // first query row and number of tokens of the block
    int h;                    // kv head; -1: no more items
    int k_row, keys;          // the sequence's first key and their number
    int last;                 // the last key that the block's first token sees (may be negative)
    int t0, t1;               // key tiles
    int whole;                // the run holds the whole block
};

struct Misc {
    uint64_t q_full[2], q_empty[2], s_full[2], p_ready[4], o_done[2], full[12], empty[12], item_full[NI], item_empty[NI],
        drain;
    Item items[NI];
    unsigned long long warp_units[THREADS / 32], total, rest;
    int first_seq, abort;
    uint32_t tmem;
};
static_assert(sizeof(Misc) <= 1024, "small area");

struct Args {
    const int32_t *q_start, *k_start;
    int n_seq, n_q, n_k, H_q, H_kv, G;
    int tok;                  // tokens of a tile: 128 / G
    void *out;
    float *lse;
    float *part_o;            // [CTA][2][256][D]
    float2 *part_ml;          // [CTA][2][256]
    int4 *desc;               // [CTA][2]: the block that this CTA begins and others finish (see combine)
    float scale_log2;
};

// ---- the list --------------------------------------------------------------------------------------------
// Sequence i's extent, safe whatever the start arrays hold: rows and keys are cut at the tensors' ends.
struct Seq {
    int q0, nq, k0, nk;
};
__device__ __forceinline__ Seq make_seq(const Args &a, int q0, int q1, int k0, int k1) {
    // queries are counted from the end of their sequence; rows past the tensor are not there, but still count
    Seq s;
    s.q0 = q0;
    s.nq = q0 < 0 || q0 >= a.n_q || q1 <= q0 ? 0 : q1 - q0;
    k0 = max(k0, 0);
    s.k0 = k0;
    s.nk = max(min(k1, a.n_k) - k0, 0);
    return s;
}
__device__ __forceinline__ Seq load_seq(const Args &a, int i) {
    return make_seq(a, __ldcg(a.q_start + i), __ldcg(a.q_start + i + 1), __ldcg(a.k_start + i), __ldcg(a.k_start + i + 1));
}
__device__ __forceinline__ int blocks_of(const Args &a, const Seq &s) {
    const int rows = min(s.nq, a.n_q - s.q0);   // rows that exist
    return s.nq > 0 ? (rows + 2 * a.tok - 1) / (2 * a.tok) : 0;
}
// keys that block b sees, at least 1 (a block without keys still writes its rows)
__device__ __forceinline__ int keys_of(const Args &a, const Seq &s, int b) {
    const long long t2 = 2 * a.tok, end = min((long long)s.nq, (b + 1) * t2) + s.nk - s.nq;
    return (int)max(min(end, (long long)s.nk), 1ll);
}
// units of the blocks before b: with off = nk - nq, a block sees off + (b + 1) t2 keys, or 1 where that is less;
// only the last, which is never summed here before the end, is cut at nk
__device__ __forceinline__ long long units_before(const Args &a, const Seq &s, int b, int blocks) {
    const long long t2 = 2 * a.tok, off = s.nk - s.nq;
    const int n = min(b, blocks - 1);                                     // blocks summed by the formula
    const long long b0 = off >= 0 ? 0 : min((long long)n, -off / t2);        // of which the first b0 see nothing
    long long u = (long long)b * BLOCK_COST + b0 + (n - b0) * off + t2 * ((long long)n * (n + 1) / 2 - b0 * (b0 + 1) / 2);
    if (b == blocks) u += keys_of(a, s, blocks - 1);
    return u;
}
__device__ __forceinline__ unsigned long long units_of(const Args &a, const Seq &s) {
    const int n = blocks_of(a, s);
    return n ? (unsigned long long)units_before(a, s, n, n) : 0;
}
__device__ __forceinline__ unsigned long long runs_of(unsigned long long W) {
    return max(min((unsigned long long)gridDim.x, W / (2 * BN)), 1ull);
}
__device__ __forceinline__ unsigned long long run_start(unsigned long long W, unsigned c) {
    const unsigned long long P = runs_of(W);
    return c >= P ? W : W * c / P;
}
// the tile of a block at which a cut `x` units into it falls
__device__ __forceinline__ int cut_tile(long long x, int tiles) {
    if (x <= BLOCK_COST) return 0;
    const int t = (int)((x - BLOCK_COST + BN - 1) / BN);
    return t < SNAP ? 0 : tiles - t < SNAP ? tiles : t;
}

// A wait of a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// MMAs with the descriptors' two words apart.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi),
        "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc),
        "r"((uint32_t)acc)
        : "memory");
}

// key tiles [t0, t1) of one of an item's two tiles: the first tile's tokens see fewer keys than the second's
__device__ __forceinline__ int tile_end(const Args &a, const Item &it, int x) {
    if (x == 1) return it.tokens > a.tok ? it.t1 : it.t0;   // no second tile
    if (it.tokens <= a.tok) return it.t1;
    const int n = min(it.last + a.tok, it.keys);             // keys that the first tile sees
    return max(min(it.t1, n > 0 ? (n + BN - 1) / BN : 1), it.t0);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    packed_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const Args a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    if (sm + C::USED > smem_raw + C::ALLOC) {  // the tiles need 1024-byte alignment
        if (threadIdx.x == 0) atomicExch(&g_packed_status, 2);
        return;
    }
    Misc *ms = reinterpret_cast<Misc *>(sm + C::OFF_MISC);
    volatile int *s_abort = &ms->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ms->abort = 0;
        for (int x = 0; x < 2; ++x) {
            mbar_init(&ms->q_full[x], 1);
            mbar_init(&ms->q_empty[x], 1);
            mbar_init(&ms->s_full[x], 1);
            mbar_init(&ms->p_ready[2 * x], 128);
            mbar_init(&ms->p_ready[2 * x + 1], 128);
            mbar_init(&ms->o_done[x], 1);
        }
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&ms->full[s], 1);
            mbar_init(&ms->empty[s], 1);
        }
        for (int s = 0; s < NI; ++s) {
            mbar_init(&ms->item_full[s], 1);
            mbar_init(&ms->item_empty[s], 9);   // MMA warp, eight softmax warps
        }
        mbar_init(&ms->drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&ms->tmem, TMEM_COLS);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    // ---- this CTA's run of the list: where it starts
    {
        const int per = (a.n_seq + THREADS - 1) / THREADS;
        const int i0 = min((int)threadIdx.x * per, a.n_seq), i1 = min(i0 + per, a.n_seq);
        unsigned long long mine = 0;
        for (int i = i0; i < i1; ++i) mine += units_of(a, load_seq(a, i));
        unsigned long long sum = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const unsigned long long up = __shfl_up_sync(0xffffffffu, sum, x);
            if (lane >= x) sum += up;
        }
        if (lane == 31) ms->warp_units[warp] = sum;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        unsigned long long before = sum - mine, total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += ms->warp_units[w];
            total += ms->warp_units[w];
        }
        unsigned long long r = total ? run_start(total * a.H_kv, blockIdx.x) % total : 0;
        if (threadIdx.x == 0) ms->total = total;
        if (r >= before && r < before + mine) {
            r -= before;
            int i = i0;
            for (; i + 1 < i1; ++i) {
                const unsigned long long n = units_of(a, load_seq(a, i));
                if (r < n) break;
                r -= n;
            }
            ms->first_seq = i;
            ms->rest = r;
        }
        __syncthreads();
    }
    const uint32_t tmem = ms->tmem;

    // registers: 128 * 88 + 256 * 208 = 384 * 168, what the CTA is launched with
    if (warp < 4) setmaxnreg_dec<88>();
    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        const unsigned long long W = ms->total * a.H_kv, u0 = run_start(W, blockIdx.x), u1 = run_start(W, blockIdx.x + 1);
        unsigned long long left = u1 - u0;
        uint32_t n_item = 0, n_ring = 0, nq[2] = {0, 0};
        bool ok = true;
        int owner_first = 0;   // this CTA begins a block that others finish
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        int seq = 0, h = 0, block = 0, blocks = 0, base = 0, held_q = 0, held_k = 0, held_q1 = 0, held_k1 = 0;
        long long x = 0;       // units of the block that lie before this run
        Seq s = {0, 0, 0, 0};
        auto hold = [&]() {    // the starts of 32 sequences from `seq`, a lane each
            base = seq;
            const int i = min(base + lane, a.n_seq - 1);
            held_q = __ldcg(a.q_start + i); held_q1 = __ldcg(a.q_start + i + 1);
            held_k = __ldcg(a.k_start + i); held_k1 = __ldcg(a.k_start + i + 1);
        };
        auto enter = [&]() {   // sequence `seq`
            if (seq < base || seq - base >= 32) hold();
            const int l = seq - base;
            s = make_seq(a, __shfl_sync(0xffffffffu, held_q, l), __shfl_sync(0xffffffffu, held_q1, l),
                         __shfl_sync(0xffffffffu, held_k, l), __shfl_sync(0xffffffffu, held_k1, l));
            blocks = blocks_of(a, s);
            block = 0;
        };
        if (left) {
            seq = ms->first_seq;
            h = (int)(u0 / ms->total);
            hold();
            enter();
            const long long r = (long long)ms->rest;
            int lo = 0, hi = blocks;   // units_before(lo) <= r < units_before(hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (units_before(a, s, mid, blocks) <= r) lo = mid; else hi = mid;
            }
            block = lo;
            x = r - units_before(a, s, lo, blocks);
        }
        while (ok && left && h < a.H_kv) {
            if (block >= blocks) {
                if (++seq == a.n_seq) { seq = 0; ++h; }
                enter();
                continue;
            }
            Item it;
            const int seen = keys_of(a, s, block), tiles = (seen + BN - 1) / BN;
            const long long all = seen + BLOCK_COST, x1 = (long long)min((unsigned long long)all, x + left);
            it.t0 = cut_tile(x, tiles);
            it.t1 = x1 == all ? tiles : cut_tile(x1, tiles);
            it.q_row = s.q0 + block * 2 * a.tok;
            it.tokens = min(2 * a.tok, min(s.nq, a.n_q - s.q0) - block * 2 * a.tok);
            it.h = h;
            it.k_row = s.k0;
            it.keys = s.nk;
            it.last = block * 2 * a.tok + s.nk - s.nq;
            it.whole = it.t0 == 0 && it.t1 == tiles;
            left -= x1 - x;
            if (it.t0 == 0 && it.t1 > 0 && it.t1 < tiles) {
                // others finish this block: those of the next runs whose cuts leave them a part of it
                owner_first = 1;
                if (lane == 0) {
                    const unsigned long long begin = u1 - x1;   // the block's first unit
                    int n = 1;
                    for (unsigned c = blockIdx.x + 1;; ++c, ++n) {
                        const unsigned long long e = run_start(W, c + 1);
                        if (e >= begin + all || cut_tile((long long)(e - begin), tiles) == tiles) { ++n; break; }
                    }
                    a.desc[2 * blockIdx.x] = make_int4(it.q_row, it.tokens, h, n);
                }
            }
            x = 0;
            ++block;
            if (it.t1 <= it.t0) continue;
            const int slot = n_item % NI;
            if (n_item >= NI && !warp_wait(&ms->item_empty[slot], ((n_item / NI) - 1) & 1, s_abort)) break;
            if (lane == 0) {
                ms->items[slot] = it;
                mbar_arrive(&ms->item_full[slot]);
            }
            ++n_item;
            auto load_kv = [&](const CUtensorMap *m, int t) -> bool {
                const int st = n_ring % C::NS;
                if (n_ring >= (uint32_t)C::NS && !warp_wait(&ms->empty[st], ((n_ring / C::NS) - 1) & 1, s_abort)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ms->full[st], C::TILE);
#pragma unroll
                    for (int dh = 0; dh < D / 64; ++dh)
                        tma_load_3d(sm + C::OFF_RING + st * C::TILE + dh * BN * 128, m, &ms->full[st], dh * 64, h, it.k_row + t * BN);
                }
                ++n_ring;
                return true;
            };
            const int two = it.tokens > a.tok ? 2 : 1;
            for (int i = 0; ok && i < two; ++i) {
                if (nq[i] > 0 && !warp_wait(&ms->q_empty[i], (nq[i] - 1) & 1, s_abort)) { ok = false; break; }
                ++nq[i];
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ms->q_full[i], (D / 64) * a.tok * a.G * 128);
#pragma unroll
                    for (int dh = 0; dh < D / 64; ++dh)
                        tma_load_3d(sm + C::OFF_Q + i * C::TILE + dh * BM * 128, &tm_q, &ms->q_full[i], dh * 64, h * a.G, it.q_row + i * a.tok);
                }
                if (i == 0) ok = load_kv(&tm_k, it.t0);   // the first product waits for these two
            }
            for (int t = it.t0; ok && t < it.t1; ++t) {
                if (t > it.t0) ok = load_kv(&tm_k, t);
                if (ok) ok = load_kv(&tm_v, t);
            }
        }
        if (!owner_first && lane == 0) a.desc[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
        if (ok) {   // the end of the items
            const int slot = n_item % NI;
            if (n_item < NI || warp_wait(&ms->item_empty[slot], ((n_item / NI) - 1) & 1, s_abort)) {
                if (lane == 0) {
                    ms->items[slot].h = -1;
                    mbar_arrive(&ms->item_full[slot]);
                }
            }
        }
        if (*s_abort) {   // a wait gave up: let the copies in flight land before the CTA exits
            volatile int never = 0;
            for (uint32_t st = 0; st < (uint32_t)C::NS && st < n_ring; ++st) {
                const uint32_t last = st + ((n_ring - 1 - st) / C::NS) * C::NS;
                mbar_wait(&ms->full[st], (last / C::NS) & 1, &never, 200000000ull);
            }
            for (int i = 0; i < 2; ++i)
                if (nq[i] > 0) mbar_wait(&ms->q_full[i], (nq[i] - 1) & 1, &never, 200000000ull);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t FMT = BF16 ? (1u << 7) | (1u << 10) : 0u;
            constexpr uint32_t IDESC_S = idesc_f16(BM, BN, 0, 0) | FMT, IDESC_O = idesc_f16(BM, D, 0, 1) | FMT;
            // descriptors: the high word is fixed, the low word is the address (in 16 bytes) under the leading offset;
            // between the steps of a product only the address moves
            constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
            const uint32_t lo_q = (smem_u32(sm + C::OFF_Q) >> 4) | (1u << 16), lo_ring = smem_u32(sm + C::OFF_RING) >> 4;
            uint32_t n_item = 0, ring = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;
            bool ok = true;
            Item it;
            // S of tile x = Q_x K^T, K in ring entry r
            auto issue_s = [&](int x, uint32_t r) {
                const uint32_t kb = (lo_ring + (r % C::NS) * (C::TILE >> 4)) | (1u << 16), qb = lo_q + x * (C::TILE >> 4);
                const uint32_t d = tmem + C::COL_S + 128 * x;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = (ks >> 2) * (128 * 128 >> 4) + (ks & 3) * 2;
                    umma_ss(d, qb + off, kb + off, DESC_HI, IDESC_S, ks > 0);
                }
                umma_commit(&ms->s_full[x]);
            };
            // half of O of tile x (+)= P_x V (keys 64 hf .. + 63 of the tile), V in ring entry r
            auto issue_pv = [&](int x, int hf, uint32_t r, bool acc) {
                const uint32_t vb = (lo_ring + (r % C::NS) * (C::TILE >> 4)) | ((BN * 128 >> 4) << 16);
                const uint32_t d = tmem + C::COL_O + D * x, pa = tmem + C::COL_S + 128 * x;
#pragma unroll
                for (int i = 0; i < BN / 32; ++i) {
                    const int ks = BN / 32 * hf + i;
                    umma_ts(d, pa + ks * 8, vb + ks * (16 * 128 >> 4), DESC_HI, IDESC_O, i > 0 || acc);
                }
            };
            auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
                const bool k = mbar_wait(bar, parity, s_abort);
                tc_fence_after();
                return k;
            };
            auto ring_wait = [&](uint32_t r) -> bool { return wait(&ms->full[r % C::NS], (r / C::NS) & 1); };
            while (ok) {
                const int slot = n_item % NI;
                if (!mbar_wait(&ms->item_full[slot], (n_item / NI) & 1, s_abort)) break;
                it = ms->items[slot];
                ++n_item;
                mbar_arrive(&ms->item_empty[slot]);
                if (it.h < 0) break;
                const int end0 = tile_end(a, it, 0), end1 = tile_end(a, it, 1);
                const bool two = it.tokens > a.tok;
                if (!(ok = ring_wait(ring))) break;
                if (!(ok = wait(&ms->q_full[0], nq0 & 1))) break;
                ++nq0;
                if (it.t0 < end0) issue_s(0, ring);
                if (it.t0 + 1 >= end0) umma_commit(&ms->q_empty[0]);   // its only product with K: Q may be replaced
                if (two) {
                    if (!(ok = wait(&ms->q_full[1], nq1 & 1))) break;
                    ++nq1;
                    issue_s(1, ring);
                    if (it.t0 + 1 >= end1) umma_commit(&ms->q_empty[1]);
                }
                umma_commit(&ms->empty[ring % C::NS]);
                for (int t = it.t0; ok && t < it.t1; ++t) {
                    const uint32_t rv = ring + 1 + 2 * (t - it.t0), rk = rv + 1;
                    const bool more = t + 1 < it.t1;
                    if (!(ok = ring_wait(rv))) break;
                    if (more && !(ok = ring_wait(rk))) break;
                    if (t < end0) {
                        if (!(ok = wait(&ms->p_ready[0], np0 & 1))) break;
                        issue_pv(0, 0, rv, t > it.t0);
                        if (!(ok = wait(&ms->p_ready[1], np0 & 1))) break;
                        issue_pv(0, 1, rv, true);
                        ++np0;
                        if (t + 1 < end0) {
                            issue_s(0, rk);
                            if (t + 2 >= end0) umma_commit(&ms->q_empty[0]);
                        } else {
                            umma_commit(&ms->o_done[0]);
                        }
                    }
                    if (t < end1) {
                        if (!(ok = wait(&ms->p_ready[2], np1 & 1))) break;
                        issue_pv(1, 0, rv, t > it.t0);
                        if (!(ok = wait(&ms->p_ready[3], np1 & 1))) break;
                        issue_pv(1, 1, rv, true);
                        ++np1;
                        if (t + 1 < end1) {
                            issue_s(1, rk);
                            if (t + 2 >= end1) umma_commit(&ms->q_empty[1]);
                        } else {
                            umma_commit(&ms->o_done[1]);
                        }
                    }
                    umma_commit(&ms->empty[rv % C::NS]);
                    if (more) umma_commit(&ms->empty[rk % C::NS]);
                }
                ring += 2 * (it.t1 - it.t0);
            }
            if (*s_abort) {   // let the MMAs in flight finish before tensor memory is freed
                volatile int never = 0;
                umma_commit(&ms->drain);
                mbar_wait(&ms->drain, 0, &never, 200000000ull);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------------ softmax, a thread for each row
        setmaxnreg_inc<208>();
        const int x = (warp - 4) >> 2;                 // tile
        const int r = (warp & 3) * 32 + lane;          // row of the tile = TMEM lane
        const int token = r / a.G, head = r - token * a.G;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + C::COL_S + 128 * x + lane_base, tO = tmem + C::COL_O + D * x + lane_base;
        const float sl2 = a.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        uint32_t n_item = 0, ns = 0, no = 0, ring = 0;
        bool ok = true;
        while (ok) {
            const int slot = n_item % NI;
            if (!warp_wait(&ms->item_full[slot], (n_item / NI) & 1, s_abort)) break;
            const Item it = ms->items[slot];
            ++n_item;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms->item_empty[slot]);
            if (it.h < 0) break;
            const int tk = x * a.tok + token;                          // token of the block
            const bool valid = token < a.tok && tk < it.tokens;
            const int last = valid ? it.last + tk : -1;                  // the last key that this row sees
            const int last0 = it.last + x * a.tok;                       // ... that the tile's first row sees
            const int end = tile_end(a, it, x), end0 = tile_end(a, it, 0);
            float m = -INFINITY, l = 0.f;
            for (int t = it.t0; t < end; ++t) {
                if (!(ok = warp_wait(&ms->s_full[x], ns & 1, s_abort))) break;
                ++ns;
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32p(tS + c * 32, s + c * 32);
                tmem_ld_wait();
                const int key0 = t * BN;
                if (key0 + BN - 1 > last0) {
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (key0 + e > last) s[e] = 0xFF800000u;   // -inf
                }
                float mx8[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) mx8[u] = __uint_as_float(s[u]);
#pragma unroll
                for (int e = 8; e < 120; e += 16) {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        mx8[u] = fmax3(mx8[u], __uint_as_float(s[e + u]), __uint_as_float(s[e + 8 + u]));
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) mx8[u] = fmaxf(mx8[u], __uint_as_float(s[120 + u]));
                const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
                const float m_new = fmaxf(m, mx * sl2);
                if (t == it.t0) {
                    m = m_new;
                } else if (__any_sync(0xffffffffu, m_new > m + RESCALE_LOG2)) {
                    // S(t) is complete, so PV(t - 1), issued before it, is too
                    const bool up = m_new > m + RESCALE_LOG2;
                    const float alpha = !up ? 1.f : m == -INFINITY ? 0.f : ex2(m - m_new);
                    if (up) m = m_new;
                    l *= alpha;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + c * 32, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(tO + c * 32, o);
                    }
                }
                // a row that sees no key so far: its scores are all -inf and give p = 0 with the offset 0
                const float m_sub = m == -INFINITY ? 0.f : m;
                const uint64_t nm2 = f2_pack(-m_sub, -m_sub);
                uint64_t rs4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[32 * c + e]), __uint_as_float(s[32 * c + e + 1])), sl2x2, nm2), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        rs4[(e >> 1) & 3] = f2_add(rs4[(e >> 1) & 3], f2_pack(x0, x1));
                        pk[e >> 1] = pack16<BF16>(x0, x1);
                    }
                    tmem_st16(tS + c * 16, pk);
                    if (c == 1) {
                        // the first half of P: its product may start
                        if ((t + 1) * BN > it.keys && (x == 0 || t >= end0)) {
                            // The rows of V behind the sequence are another's or nobody's, and a NaN times a zero weight
                            // would be a NaN: the tile whose PV comes first zeroes them.  (The barrier cannot be a phase
                            // further: it is that PV that frees the ring entry.)
                            const uint32_t rv = ring + 1 + 2 * (t - it.t0);
                            ok = warp_wait(&ms->full[rv % C::NS], (rv / C::NS) & 1, s_abort);
                            uint8_t *vt = sm + C::OFF_RING + (rv % C::NS) * C::TILE;
                            for (int i = max(it.keys - t * BN, 0) * 8 + r; ok && i < BN * 8; i += BM)
#pragma unroll
                                for (int dh = 0; dh < D / 64; ++dh)
                                    *reinterpret_cast<uint4 *>(vt + dh * BN * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                            fence_proxy_async_smem();
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&ms->p_ready[2 * x]);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&ms->p_ready[2 * x + 1]);
                float r8[8];
#pragma unroll
                for (int u = 0; u < 4; ++u) f2_unpack(rs4[u], r8[2 * u], r8[2 * u + 1]);
                l += ((r8[0] + r8[1]) + (r8[2] + r8[3])) + ((r8[4] + r8[5]) + (r8[6] + r8[7]));
                if (!ok) break;
            }
            ring += 2 * (it.t1 - it.t0);
            if (!ok) break;
            // ---- O / l, or the partial.  The next item's first PV overwrites O only after this thread's next P,
            // which comes after these reads.
            if (x == 1 && it.tokens <= a.tok) continue;   // no second tile
            const bool any = it.t0 < end;
            if (any) {
                if (!(ok = warp_wait(&ms->o_done[x], no & 1, s_abort))) break;
                ++no;
                tc_fence_after();
            }
            const int64_t row = (int64_t)(it.q_row + tk) * a.H_q + it.h * a.G + head;
            const int64_t prow = ((int64_t)blockIdx.x * 2 + (it.t0 == 0)) * 256 + x * BM + r;
            const bool none = !any || l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                __syncwarp();
                if (any) {
                    tmem_ld32(tO + c, o);
                    tmem_ld_wait();
                }
                if (!valid) continue;
                if (it.whole) {
                    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out) + row * (D / 2) + c / 2;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = none ? 0u : pack16<BF16>(__uint_as_float(o[e + 2 * j]) * inv, __uint_as_float(o[e + 2 * j + 1]) * inv);
                        *reinterpret_cast<uint4 *>(dst + e / 2) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (any) {
                    uint32_t *dst = reinterpret_cast<uint32_t *>(a.part_o) + prow * D + c;
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4 *>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            __syncwarp();
            tc_fence_before();
            if (valid) {
                if (!it.whole) a.part_ml[prow] = any ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
                else if (a.lse) a.lse[row] = none ? -INFINITY : (m + log2f(l)) * LN2;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *s_abort) atomicExch(&g_packed_status, 1);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Joins the partials of the block that CTA blockIdx.x of the first kernel began: for each row
// out = sum_p w_p O_p / sum_p w_p l_p, w_p = 2^(m_p - max m), the runs in order.  D / 4 threads for a row.
constexpr int COMBINE_THREADS = 256;
constexpr int COMBINE_ROWS = 32;
template <int D, bool BF16>
__global__ void __launch_bounds__(COMBINE_THREADS) packed_combine_kernel(const Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int4 d = __ldcg(a.desc + 2 * blockIdx.x);   // first query row, tokens, kv head, partials
    if (d.w == 0) return;
    constexpr int LANES = D / 4, RPB = COMBINE_THREADS / LANES;
    const int lane = threadIdx.x % LANES;
    for (int i = threadIdx.x / LANES; i < COMBINE_ROWS; i += RPB) {
        const int r = blockIdx.y * COMBINE_ROWS + i, x = r / BM, rr = r - x * BM;
        const int token = rr / a.G, head = rr - token * a.G, tk = x * a.tok + token;
        if (token >= a.tok || tk >= d.y) continue;
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < d.w; ++p) {
            const int64_t prow = ((int64_t)(blockIdx.x + p) * 2 + (p == 0)) * 256 + r;
            const float2 ml = __ldcg(a.part_ml + prow);
            if (ml.x == -INFINITY) continue;
            const float4 o = __ldcg(reinterpret_cast<const float4 *>(a.part_o + prow * D) + lane);
            const float mx = fmaxf(m, ml.x), f = m == -INFINITY ? 0.f : ex2(m - mx), w = ex2(ml.x - mx);
            m = mx;
            l = l * f + ml.y * w;
            acc.x = acc.x * f + o.x * w; acc.y = acc.y * f + o.y * w;
            acc.z = acc.z * f + o.z * w; acc.w = acc.w * f + o.w * w;
        }
        const int64_t row = (int64_t)(d.x + tk) * a.H_q + d.z * a.G + head;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        reinterpret_cast<uint2 *>(a.out)[row * LANES + lane] =
            make_uint2(pack16<BF16>(acc.x * inv, acc.y * inv), pack16<BF16>(acc.z * inv, acc.w * inv));
        if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
}

template <int D, bool BF16>
int launch_t(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, int ctas, cudaStream_t s) {
    if (allow_dynamic_smem((const void *)packed_kernel<D, BF16>, Cfg<D>::ALLOC) != KVC_OK) return KVC_ECUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Cfg<D>::ALLOC;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, packed_kernel<D, BF16>, tq, tk, tv, a) != cudaSuccess) return KVC_ECUDA;
    cfg.gridDim = dim3(ctas, 2 * BM / COMBINE_ROWS);
    cfg.blockDim = dim3(COMBINE_THREADS);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, packed_combine_kernel<D, BF16>, a) != cudaSuccess) return KVC_ECUDA;
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ECUDA;
}

}  // namespace

size_t packed_scratch_bytes(int, int, int, int, int head_dim) {
    return (size_t)sm_count() * (2 * sizeof(int4) + 2 * 256 * (head_dim * sizeof(float) + sizeof(float2)));
}

int launch_packed(const PackedArgs &p, void *scratch, cudaStream_t s) {
    const int ctas = sm_count();
    Args a;
    a.q_start = p.q_start;
    a.k_start = p.k_start;
    a.n_seq = p.n_seq;
    a.n_q = p.n_q;
    a.n_k = p.n_k;
    a.H_q = p.H_q;
    a.H_kv = p.H_kv;
    a.G = p.H_q / p.H_kv;
    a.tok = BM / a.G;
    a.out = p.out;
    a.lse = p.lse;
    a.desc = static_cast<int4 *>(scratch);
    a.part_o = reinterpret_cast<float *>(a.desc + 2 * ctas);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)ctas * 2 * 256 * p.D);
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)p.D);
    const bool bf = p.dtype == KVC_IN_BF16;
    const CUtensorMapDataType dt = bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap tq, tk, tv;
    const bool none = p.n_k == 0;   // no keys: the maps of K and V are never loaded from a row that exists
    auto map = [&](CUtensorMap *m, const void *base, int heads, int rows, int64_t ld, int box_heads, int box_rows) {
        return make_map_3d(m, dt, base, p.D, heads, rows, (uint64_t)p.D * 2, (uint64_t)ld * 2, 64, box_heads, box_rows,
                           CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!map(&tq, p.q, p.H_q, p.n_q, p.ld_q, a.G, a.tok) ||
        !map(&tk, none ? p.q : p.k, p.H_kv, none ? 1 : p.n_k, none ? p.ld_q : p.ld_k, 1, BN) ||
        !map(&tv, none ? p.q : p.v, p.H_kv, none ? 1 : p.n_k, none ? p.ld_q : p.ld_v, 1, BN))
        return KVC_ECUDA;
    if (p.D == 128) return bf ? launch_t<128, true>(tq, tk, tv, a, ctas, s) : launch_t<128, false>(tq, tk, tv, a, ctas, s);
    return bf ? launch_t<64, true>(tq, tk, tv, a, ctas, s) : launch_t<64, false>(tq, tk, tv, a, ctas, s);
}

int read_and_clear_packed_status(int32_t *status) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_packed_status, sizeof(int)) != cudaSuccess) return KVC_ECUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_packed_status, &zero, sizeof(int)) != cudaSuccess) return KVC_ECUDA;
    *status = v;
    return KVC_OK;
}

}  // namespace kvc
