// Causal attention of packed prompts with grouped heads, on the fifth-generation tensor cores.
//
// Sequence s has nq query rows and nk keys; row i sees the keys j <= i + nk - nq:
//   out[i][h] = sum_j softmax_j(q[i][h] . k[j][h/G] / sqrt(D)) v[j][h/G].
// Both products are contractions of the inputs' own type (bf16 or fp16) with float32 accumulators in tensor
// memory; the softmax runs in one pass over the keys with the row's running maximum and sum in float32; its
// numerators are rounded to the inputs' type for the second product.  What bounds long prompts is the softmax
// warps' chain of each tile (below), and short ones the chain load - product - softmax - product - store of
// each block.
//
// Measured (of the rate of a large matrix product): one prompt of 10,041 tokens, 40 query and 8 kv heads of 128, 797 us
// (1,295 TF/s, 0.67); 48 prompts of 1 to 513 tokens 60 us; 512-token chunks over prefixes of 2,500 to 9,000, 16
// and 4 heads of 64, 79 us (600 TF/s, 0.31).  The long prompt with parts of the work left out: neither loads, products nor
// softmax (the barriers, tensor memory's loads and stores) 363 us, loads alone 509, products alone 590, both 640, all
// but the products 718.  The softmax's arithmetic and the waits around it hardly overlap, since all of a CTA's softmax
// warps are in the same phase; and the GPU is at its power limit (1400 W; the clock falls from 2.07 to 1.75-1.95 GHz),
// so that eight softmax warps of 128 keys each, or sixteen, or two sets of eight all take 790 to 830 us.
//
// Work split.  The G query heads of a kv head see the same keys, so a block of 128 rows holds 128 / G tokens with all
// their heads: a prompt of 25 tokens with five heads fills one block where a block for each head would leave four
// fifths of five empty.  The blocks of all kv heads and sequences, each as long as the keys that it sees plus a
// charge, form one list that is cut into equal runs, one for each CTA (one per SM); lengths are read on the device.  A
// block cut by a run's end leaves partial results (O, maximum, sum; at most two blocks for each CTA) that a second
// kernel joins in the runs' order; cuts close to a block's end move there.
//
// Tensor memory (512 columns): S = Q K^T of a tile of 256 keys (256 columns), P (its softmax numerators as 16-bit pairs,
// 128 columns) and O (D).  S and P are apart, so S of the next tile - of the next block, at a block's end - is computed
// while the softmax of this one runs.  What a tile costs beside its arithmetic - waits, loads from tensor memory, the
// exchange of maxima, about 1,500 cycles - is why a tile has 256 keys.  Two sets of eight softmax warps that take tiles
// of 128 keys in turn, S and P in two buffers each, so that one set's waits are the other's arithmetic, took 808 us
// for the long prompt, 63 for the short ones and 74 for the chunks.
//
// One CTA (20 warps):
//   warp 0     producer: walks the CTA's run of the list, passes each block on through a ring of items and
//              loads Q (two buffers) and K and V (a ring each of 128-key pieces), in the order K(0) K(1) V(0) K(2) V(1)
//              ..., by TMA;
//   warps 1, 2   one lane of each issues the MMAs: those with K, and those with V (one thread for both spends as long in their
//              waits and commits, about 100 and 60 cycles each, as the tensor cores on the products); warp 1 also
//              allocates tensor memory;
//   warps 4-19  softmax, four threads for each row, 64 keys of each tile each, 32 of either half.  They exchange their
//              maxima through shared memory, but go on with the reference that the row has: it is raised, and O rescaled,
//              only where a score passes it by more than 2^8 (fp16: 2^15, a raised reference lying 2^7 below the maximum).
//              Where a sequence ends inside a piece of V these warps also set the rows behind it to zero.
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

constexpr int BM = 128;             // rows of a block
constexpr int BN = 256;             // keys of a tile
constexpr int HN = 128;             // keys of half a tile
constexpr int GROUPS = 4;           // softmax threads of a row
constexpr int THREADS = 128 * (1 + GROUPS);
constexpr int NI = 4;               // items on their way from the producer
// What a block costs besides its keys, in keys.  With 256, 384, 512 and 1,024 the long prompt above takes 865, 839, 797 and
// 798 us, the short ones 63.6, 60.6, 59.8 and 62.4.
constexpr int BLOCK_COST = 512;
// A cut fewer tiles than this from an end of a block moves there.  With 1, 2 and 4 the short prompts take 65.9, 59.8 and
// 61.2 us, the chunks 77.4, 77.6 and 80.7.
constexpr int SNAP = 2;
constexpr int MAX_DYN_SMEM = 232448;
// A row's reference lies this far below its greatest score: with fp16 numerators 2^7, so that numerators (2^15 at most before
// the reference is raised) are held down to 2^-31 of the greatest.  With the reference at the score itself those below 2^-25
// vanished from O, but not from the sum.  bf16 has the range.  Less log2(2 / 1.9375), as the greatest numerator is often most of
// a row's sum: it then lies just below a power of two (up to scores of 64 the reference misses by 3/64 at most), where a
// rounding is half as coarse, relative to the number, as just above one; 1.9375 is a number that both types hold.  Error
// against 64 bits, of that of rounding the output alone, prompts of 2, 8 and 500 tokens: fp16 1.22, 1.26 and 1.33 instead of
// 1.79, 1.50 and 1.48 with 7, bf16 1.11, 1.18 and 1.30 instead of 1.12, 1.18 and 1.33 with 0.
template <bool BF16>
constexpr float SHIFT_LOG2 = (BF16 ? 0.0f : 7.0f) - 0.045803690f;
template <bool BF16>
constexpr float RESCALE_LOG2 = SHIFT_LOG2<BF16> + 8.0f;
constexpr float LN2 = 0.69314718055994531f;
constexpr uint32_t TMEM_COLS = 512;

template <int D>
struct Cfg {
    static constexpr int PIECE = 128 * D * 2;              // 128 rows of Q, K or V
    static constexpr int KS = D == 128 ? 3 : 6, VS = D == 128 ? 2 : 5;   // pieces of K and V on their way
    static constexpr int OFF_Q = 0, OFF_K = 2 * PIECE, OFF_V = OFF_K + KS * PIECE, OFF_MISC = OFF_V + VS * PIECE;
    static constexpr int OFF_MAIL = OFF_MISC + 1024;
    static constexpr int USED = OFF_MAIL + 2 * BM * GROUPS * 2;
    static constexpr int ALLOC = USED + 1024 <= MAX_DYN_SMEM ? USED + 1024 : MAX_DYN_SMEM;
    static_assert(USED <= MAX_DYN_SMEM, "shared memory plan");
};
constexpr uint32_t COL_S = 0, COL_P = 256, COL_O = 384;

// A block, or the part of its keys that falls into this CTA's run.
struct Item {
    int q_row, tokens;        // first query row and number of tokens of the block
    int h;                    // kv head; -1: no more items
    int k_row, keys;          // the sequence's first key and their number
    int last;                 // the last key that the block's first token sees (may be negative, -BM at least)
    int seen;                 // keys that the block sees, at least 1
    int t0, t1;               // key tiles
    int whole;                // the run holds the whole block
};
// halves of tile t that the block sees something of: 1 or 2
__device__ __forceinline__ int halves(int seen, int t) { return seen - t * BN > HN ? 2 : 1; }

struct Misc {
    uint64_t q_full[2], q_empty[2], s_full, s_free, p_ready, o_done, k_full[6], k_empty[6], v_full[6], v_empty[6], item_full[NI], item_empty[NI], drain[2], stall;
    Item items[NI];
    unsigned long long warp_units[THREADS / 32], total, rest;
    int first_seq, abort;
    uint32_t tmem, k_pieces, v_pieces, q_tiles;   // the last three: what the producer has asked for in all
};
static_assert(sizeof(Misc) <= 1024, "small area");

struct Args {
    const int32_t *q_start, *k_start;
    int n_seq, n_q, n_k, H_q, H_kv, G;
    int tok;                  // tokens of a block: 128 / G
    void *out;
    float *lse;
    float *part_o;            // [CTA][2][128][D]
    float2 *part_ml;          // [CTA][2][128]
    int4 *desc;               // [CTA]: the block that this CTA begins and others finish (see combine)
    float scale_log2;
    uint64_t stall_ns;        // test hook: > 0 makes the thread that issues the products with V wait for what never comes
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
    k1 = min(k1, a.n_k);
    s.nk = k1 > k0 ? k1 - k0 : 0;   // (a difference of any two numbers could pass 32 bits)
    s.k0 = s.nk ? k0 : 0;
    return s;
}
__device__ __forceinline__ Seq load_seq(const Args &a, int i) {
    return make_seq(a, __ldcg(a.q_start + i), __ldcg(a.q_start + i + 1), __ldcg(a.k_start + i), __ldcg(a.k_start + i + 1));
}
__device__ __forceinline__ int blocks_of(const Args &a, const Seq &s) {
    const int rows = min(s.nq, a.n_q - s.q0);   // rows that exist
    return s.nq > 0 ? (rows + a.tok - 1) / a.tok : 0;
}
// keys that block b sees, at least 1 (a block without keys still writes its rows)
__device__ __forceinline__ int keys_of(const Args &a, const Seq &s, int b) {
    const long long t2 = a.tok, end = min((long long)s.nq, (b + 1) * t2) + s.nk - s.nq;
    return (int)max(min(end, (long long)s.nk), 1ll);
}
// units of the blocks before b: with off = nk - nq, a block sees off + (b + 1) t2 keys, or 1 where that is less;
// only the last, which is never summed here before the end, is cut at nk
__device__ __forceinline__ long long units_before(const Args &a, const Seq &s, int b, int blocks) {
    const long long t2 = a.tok, off = s.nk - s.nq;
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

// One arrival for a whole warp, behind what all its lanes did (32 arrivals on one word are taken one by one).
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
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

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    packed_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const Args a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    if (sm + C::USED > smem_raw + C::ALLOC) {  // the tiles need 1024-byte alignment: nothing is computed, nothing joined
        asm volatile("griddepcontrol.wait;" ::: "memory");   // who waits for this kernel waits for those before it too
        if (threadIdx.x == 0) {
            a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
            atomicExch(&g_packed_status, 2);
        }
        return;
    }
    Misc *ms = reinterpret_cast<Misc *>(sm + C::OFF_MISC);
    volatile int *s_abort = &ms->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < BM * GROUPS; i += THREADS) reinterpret_cast<uint32_t *>(sm + C::OFF_MAIL)[i] = 0x00010001u;
    if (threadIdx.x == 0) {
        ms->abort = 0;
        for (int x = 0; x < 2; ++x) {
            mbar_init(&ms->q_full[x], 1);
            mbar_init(&ms->q_empty[x], 4 * GROUPS);
        }
        mbar_init(&ms->s_free, 4 * GROUPS);
        mbar_init(&ms->s_full, 1);
        mbar_init(&ms->p_ready, 4 * GROUPS);
        mbar_init(&ms->o_done, 1);
        for (int s = 0; s < 6; ++s) {
            mbar_init(&ms->k_full[s], 1);
            mbar_init(&ms->k_empty[s], 1);
            mbar_init(&ms->v_full[s], 1);
            mbar_init(&ms->v_empty[s], 1);
        }
        for (int s = 0; s < NI; ++s) {
            mbar_init(&ms->item_full[s], 1);
            mbar_init(&ms->item_empty[s], 2 + 4 * GROUPS);   // the MMA issuers and the softmax warps
        }
        mbar_init(&ms->drain[0], 1);
        mbar_init(&ms->drain[1], 1);
        mbar_init(&ms->stall, 1);
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

    // registers: 128 * 64 + 512 * 104 = 640 * 96, what the CTA is launched with
    if (warp < 4) setmaxnreg_dec<64>();
    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        const unsigned long long W = ms->total * a.H_kv, u0 = run_start(W, blockIdx.x), u1 = run_start(W, blockIdx.x + 1);
        unsigned long long left = u1 - u0;
        uint32_t n_item = 0, n_k = 0, n_v = 0, nq = 0;
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
        // the next item of the run, or h = -1
        auto next_item = [&](Item &it) {
            it.h = -1;
            while (left && h < a.H_kv) {
                if (block >= blocks) {
                    if (++seq == a.n_seq) { seq = 0; ++h; }
                    enter();
                    continue;
                }
                const int seen = keys_of(a, s, block), tiles = (seen + BN - 1) / BN;
                const long long all = seen + BLOCK_COST, x1 = (long long)min((unsigned long long)all, x + left);
                it.t0 = cut_tile(x, tiles);
                it.t1 = x1 == all ? tiles : cut_tile(x1, tiles);
                it.q_row = s.q0 + block * a.tok;
                it.tokens = min(a.tok, min(s.nq, a.n_q - s.q0) - block * a.tok);
                it.k_row = s.k0;
                it.keys = s.nk;
                it.seen = seen;
                it.last = max(block * a.tok + s.nk - s.nq, -BM);   // (no token of the block then sees anything either way)
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
                        a.desc[blockIdx.x] = make_int4(it.q_row, it.tokens, h, n);
                    }
                }
                x = 0;
                ++block;
                if (it.t1 > it.t0) {
                    it.h = h;
                    return;
                }
            }
        };
        auto publish = [&](const Item &it) -> bool {
            const int slot = n_item % NI;
            if (n_item >= NI && !warp_wait(&ms->item_empty[slot], ((n_item / NI) - 1) & 1, s_abort)) return false;
            if (lane == 0) {
                ms->items[slot] = it;
                mbar_arrive(&ms->item_full[slot]);
            }
            ++n_item;
            return true;
        };
        auto load_piece = [&](const CUtensorMap *m, uint8_t *ring, uint64_t *full, uint64_t *empty, int slots, uint32_t &n,
                              const Item &i, int key) -> bool {
            const int st = n % slots;
            if (n >= (uint32_t)slots && !warp_wait(&empty[st], ((n / slots) - 1) & 1, s_abort)) return false;
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[st], C::PIECE);
#pragma unroll
                for (int dh = 0; dh < D / 64; ++dh)
                    tma_load_3d(ring + st * C::PIECE + dh * HN * 128, m, &full[st], dh * 64, i.h, i.k_row + key);
            }
            ++n;
            return true;
        };
        auto load_k = [&](const Item &i, int t) -> bool {   // the second half first
            for (int x = halves(i.seen, t) - 1; x >= 0; --x)
                if (!load_piece(&tm_k, sm + C::OFF_K, ms->k_full, ms->k_empty, C::KS, n_k, i, t * BN + x * HN)) return false;
            return true;
        };
        auto load_v = [&](const Item &i, int t) -> bool {
            for (int x = 0; x < halves(i.seen, t); ++x)
                if (!load_piece(&tm_v, sm + C::OFF_V, ms->v_full, ms->v_empty, C::VS, n_v, i, t * BN + x * HN)) return false;
            return true;
        };
        Item it, nx;
        next_item(it);
        ok = publish(it);
        auto load_q = [&](const Item &q) -> bool {
            const int i = nq & 1;
            if (nq >= 2 && !warp_wait(&ms->q_empty[i], ((nq >> 1) - 1) & 1, s_abort)) return false;
            ++nq;
            if (lane == 0) {
                mbar_arrive_expect_tx(&ms->q_full[i], (D / 64) * a.tok * a.G * 128);
#pragma unroll
                for (int dh = 0; dh < D / 64; ++dh)
                    tma_load_3d(sm + C::OFF_Q + i * C::PIECE + dh * BM * 128, &tm_q, &ms->q_full[i], dh * 64, q.h * a.G, q.q_row);
            }
            return true;
        };
        if (ok && it.h >= 0) ok = load_q(it) && load_k(it, it.t0);
        while (ok && it.h >= 0) {
            for (int t = it.t0; ok && t + 1 < it.t1; ++t) ok = load_k(it, t + 1) && load_v(it, t);
            if (!ok) break;
            next_item(nx);   // the next block's first product comes before this one's last
            ok = publish(nx);
            if (ok && nx.h >= 0) ok = load_q(nx) && load_k(nx, nx.t0);
            if (ok) ok = load_v(it, it.t1 - 1);
            it = nx;
        }
        if (!owner_first && lane == 0) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        if (lane == 0) {
            ms->k_pieces = n_k;
            ms->v_pieces = n_v;
            ms->q_tiles = nq;
        }
    } else if (warp == 1 || warp == 2) {
        // ------------------------------------------------------------------ MMA issuers
        // Warp 1 issues the products with K, warp 2 those with V.
        if (lane == 0) {
            constexpr uint32_t FMT = BF16 ? (1u << 7) | (1u << 10) : 0u;
            constexpr uint32_t IDESC_S = idesc_f16(BM, HN, 0, 0) | FMT, IDESC_O = idesc_f16(BM, D, 0, 1) | FMT;
            // descriptors: the high word is fixed, the low word is the address (in 16 bytes) under the leading offset;
            // between the steps of a product only the address moves
            constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
            const uint32_t lo_q = (smem_u32(sm + C::OFF_Q) >> 4) | (1u << 16), lo_k = (smem_u32(sm + C::OFF_K) >> 4) | (1u << 16);
            const uint32_t lo_v = (smem_u32(sm + C::OFF_V) >> 4) | ((HN * 128 >> 4) << 16);
            uint32_t n = 0, parity = 0;           // the tile, and the parity of the ring's phase
            int slot = 0;
            bool ok = true;
            for (uint32_t n_item = 0; ok; ++n_item) {
                const int sl = n_item % NI;
                if (!mbar_wait(&ms->item_full[sl], (n_item / NI) & 1, s_abort)) break;
                const int h = ms->items[sl].h, t0 = ms->items[sl].t0, t1 = ms->items[sl].t1, seen = ms->items[sl].seen;
                mbar_arrive(&ms->item_empty[sl]);
                if (h < 0) break;
                if (warp == 1) {
                    const int qb = n_item & 1;
                    const uint32_t q = lo_q + qb * (C::PIECE >> 4);
                    if (!mbar_wait(&ms->q_full[qb], (n_item >> 1) & 1, s_abort)) break;
                    for (int t = t0; ok && t < t1; ++t, ++n) {
#pragma unroll 1
                        for (int x = halves(seen, t) - 1; x >= 0; --x) {
                            // the piece has landed, and the softmax has read what lay in this half of S
                            if (!(ok = mbar_wait(&ms->k_full[slot], parity, s_abort))) break;
                            if (n > 0 && !(ok = mbar_wait(&ms->s_free, (n - 1) & 1, s_abort))) break;
                            tc_fence_after();
                            const uint32_t kb = lo_k + slot * (C::PIECE >> 4), d = tmem + COL_S + HN * x;
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks) {
                                const uint32_t off = (ks >> 2) * (128 * 128 >> 4) + (ks & 3) * 2;
                                umma_ss(d, q + off, kb + off, DESC_HI, IDESC_S, ks > 0);
                            }
                            if (x == 0) umma_commit(&ms->s_full);
                            umma_commit(&ms->k_empty[slot]);
                            if (++slot == C::KS) { slot = 0; parity ^= 1; }
                        }
                    }
                } else {
                    if (a.stall_ns != 0) {   // gives up with S MMAs and copies in flight
                        mbar_wait(&ms->stall, 0, s_abort, a.stall_ns);
                        break;
                    }
                    for (int t = t0; ok && t < t1; ++t, ++n) {
                        const int e = halves(seen, t);
#pragma unroll 1
                        for (int x = 0; x < e; ++x) {
                            if (!(ok = mbar_wait(&ms->v_full[slot], parity, s_abort))) break;
                            if (x == 0 && !(ok = mbar_wait(&ms->p_ready, n & 1, s_abort))) break;
                            tc_fence_after();
                            const uint32_t vb = lo_v + slot * (C::PIECE >> 4);
#pragma unroll
                            for (int ks = 0; ks < HN / 16; ++ks)
                                umma_ts(tmem + COL_O, tmem + COL_P + 64 * x + ks * 8, vb + ks * (16 * 128 >> 4), DESC_HI, IDESC_O,
                                        ks > 0 || x > 0 || t > t0);
                            if (x + 1 == e) umma_commit(&ms->o_done);
                            umma_commit(&ms->v_empty[slot]);
                            if (++slot == C::VS) { slot = 0; parity ^= 1; }
                        }
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------------ softmax, four threads for each row
        setmaxnreg_inc<104>();
        const int grp = (warp - 4) >> 2;               // keys 32 grp .. + 31 of each half
        const int r = (warp & 3) * 32 + lane;          // row of the block = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + COL_S + 32 * grp + lane_base, tP = tmem + COL_P + 16 * grp + lane_base;
        const uint32_t tO = tmem + COL_O + D / GROUPS * grp + lane_base;
        const float sl2 = a.scale_log2;
        // token of the block (one that no block has, for rows behind its last) and place among its rows of the output
        const int token = r / a.G < a.tok ? r / a.G : INT32_MAX, row_off = r / a.G * a.H_q + r % a.G;
        uint32_t n = 0, n_v = 0, n_mail = 0;           // tiles, pieces of V, exchanges
        bool ok = true;
        // The four threads of a row exchange 15 bits each through shared memory; the 16th is a flag that alternates, so that
        // a word says by itself that it is new.  Two sets of words are used in turn: one is written again only after all
        // four have posted to the other, which each does after reading this one.  All read the same four words, so they
        // agree exactly.  The wait is bounded.
        const uint32_t mail = smem_u32(sm + C::OFF_MAIL) + r * (2 * GROUPS);
        auto post = [&](uint32_t bits) {
            const uint16_t w = (uint16_t)((bits & 0xFFFEu) | ((n_mail >> 1) & 1u));
            asm volatile("st.volatile.shared.b16 [%0], %1;" ::"r"(mail + (n_mail & 1u) * (BM * GROUPS * 2) + 2 * grp), "h"(w) : "memory");
        };
        auto receive = [&](uint32_t &w0, uint32_t &w1) -> bool {
            const uint32_t flags = ((n_mail >> 1) & 1u) * 0x00010001u, at = mail + (n_mail & 1u) * (BM * GROUPS * 2);
            ++n_mail;
            bool here = false;
            for (uint32_t i = 0;; ++i) {
                asm volatile("ld.volatile.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(at) : "memory");
                here = (((w0 ^ flags) | (w1 ^ flags)) & 0x00010001u) == 0;
                if (here) break;
                if ((i & 1023u) == 1023u && (*s_abort || i > (1u << 26))) {
                    *s_abort = 1;
                    break;
                }
            }
            return __all_sync(0xffffffffu, here);
        };
        // The maximum of four values, as fp16 without the last bit: the values are exponents relative to the row's reference,
        // which may be any number not far from their maximum.  -infinity travels as the lowest number.  Up to 1,024 an
        // fp16 step is 1/2, so that the rounding (half a step) and the flag in place of the last bit (one) miss a value by
        // 3/4 at most; from 16,384 on it would be 24, more than the range of fp16 numerators allows.
        auto maximum4 = [&](float v, float &all) -> bool {
            uint32_t w0, w1;
            post(__half_as_ushort(__float2half_rn(fminf(fmaxf(v, -65000.f), 65000.f))));
            const bool k = receive(w0, w1);
            const __half2 mx = __hmax2(*reinterpret_cast<__half2 *>(&w0), *reinterpret_cast<__half2 *>(&w1));
            all = fmaxf(__low2float(mx), __high2float(mx));
            return k;
        };
        // The same of any four values, all their bits, in three exchanges.
        auto maximum4_exact = [&](float v, float &all) -> bool {
            const uint32_t u = __float_as_uint(v);
            uint32_t b[4] = {0u, 0u, 0u, 0u};
            bool k = true;
#pragma unroll 1
            for (int i = 0; i < 3; ++i) {   // bits 31 to 17, 16 to 2, 1 and 0
                uint32_t w0, w1;
                post(i == 0 ? u >> 16 : i == 1 ? u >> 1 : u << 14);
                k = receive(w0, w1) && k;
                const uint32_t w[4] = {w0 & 0xFFFEu, w0 >> 16 & 0xFFFEu, w1 & 0xFFFEu, w1 >> 16 & 0xFFFEu};
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] |= i == 0 ? w[j] << 16 : i == 1 ? w[j] << 1 : w[j] >> 14;
            }
            all = fmaxf(fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1])), fmaxf(__uint_as_float(b[2]), __uint_as_float(b[3])));
            return k;
        };
        // The sum of four float32, in the groups' order, in two exchanges: all but the last two bits of each.
        auto sum4 = [&](float v, float &all) -> bool {
            const uint32_t u = __float_as_uint(v);
            uint32_t h0, h1, l0, l1;
            post(u >> 16);
            bool k = receive(h0, h1);
            post(u >> 1);
            k = receive(l0, l1) && k;
            auto join = [](uint32_t h, uint32_t lo) { return __uint_as_float((h & 0xFFFEu) << 16 | (lo & 0xFFFEu) << 1); };
            all = ((join(h0, l0) + join(h0 >> 16, l0 >> 16)) + join(h1, l1)) + join(h1 >> 16, l1 >> 16);
            return k;
        };
        constexpr float FAR = 1024.f;   // a reference is set from what maximum4 tells only between -FAR and FAR
        for (uint32_t n_item = 0; ok; ++n_item) {
            // the item stays in its slot until the block is done
            if (!warp_wait(&ms->item_full[n_item % NI], (n_item / NI) & 1, s_abort)) break;
            const volatile Item &it = const_cast<const volatile Item &>(ms->items[n_item % NI]);
            if (it.h < 0) break;
            const int t0 = it.t0, t1 = it.t1, first_last = it.last;
            int last;       // the last key that this row sees
            bool valid;
            valid = token < it.tokens;
            last = valid ? first_last + token : -1;
            // the row's reference: numerators are 2^(s sl2 - m), at most 2^8 (fp16: 2^15).  Rows that do not exist need none.
            float m = valid ? -INFINITY : 0.f, l = 0.f;
            // keys that the row does not see get -infinity
            auto mask = [&](uint32_t (&s)[32], int key0) {
                if (__builtin_expect(key0 + 31 > first_last, 0)) {
                    const int lim = last - key0;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (e > lim) s[e] = 0xFF800000u;
                }
            };
            auto maximum = [&](const uint32_t (&s)[32], float from) {
                float m4[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) m4[u] = fmax3(__uint_as_float(s[u]), __uint_as_float(s[4 + u]), __uint_as_float(s[8 + u]));
#pragma unroll
                for (int e = 12; e < 28; e += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        m4[u] = fmax3(m4[u], __uint_as_float(s[e + u]), __uint_as_float(s[e + 4 + u]));
#pragma unroll
                for (int u = 0; u < 4; ++u) m4[u] = fmaxf(m4[u], __uint_as_float(s[28 + u]));
                return fmaxf(fmax3(m4[0], m4[1], m4[2]), fmaxf(m4[3], from));
            };
            // numerators in place: the first 16 words become the pairs; their sum is added to l
            auto numerators = [&](uint32_t (&s)[32]) {
                const float m_sub = m == -INFINITY ? 0.f : m;
                const uint64_t nm2 = f2_pack(-m_sub, -m_sub), sl2x2 = f2_pack(sl2, sl2);
                uint64_t rs2[2] = {0ull, 0ull};
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sl2x2, nm2), x0, x1);
                    x0 = ex2(x0);
                    x1 = ex2(x1);
                    rs2[(e >> 1) & 1] = f2_add(rs2[(e >> 1) & 1], f2_pack(x0, x1));
                    s[e >> 1] = pack16<BF16>(x0, x1);
                }
                float r4[4];
                f2_unpack(rs2[0], r4[0], r4[1]);
                f2_unpack(rs2[1], r4[2], r4[3]);
                l += (r4[0] + r4[1]) + (r4[2] + r4[3]);
            };
            for (int t = t0; t < t1; ++t, ++n) {
                if (!(ok = warp_wait(&ms->s_full, n & 1, s_abort))) break;
                tc_fence_after();
                const bool both = halves(it.seen, t) == 2;
                uint32_t s0[32], s1[32];           // this thread's scores of either half
                tmem_ld32p(tS, s0);
                if (both) tmem_ld32p(tS + HN, s1);
                tmem_ld_wait();
                tc_fence_before();
                arrive_warp(&ms->s_free);
                mask(s0, t * BN + 32 * grp);
                float mx = maximum(s0, -INFINITY);
                if (both) {
                    mask(s1, t * BN + HN + 32 * grp);
                    mx = maximum(s1, mx);
                }
                // how far the scores pass the reference
                const bool fresh = m == -INFINITY;
                const float m_sub = fresh ? 0.f : m;
                if (!valid) mx = -INFINITY;   // rows that do not exist hold anything
                float up;
                if (!(ok = maximum4(mx * sl2 - m_sub, up))) break;
                if (__builtin_expect(__any_sync(0xffffffffu, fresh || up > RESCALE_LOG2<BF16>), 0)) {
                    // the reference rises, or is set
                    const bool told = up < FAR && (!fresh || up > -FAR);
                    if (!__all_sync(0xffffffffu, told)) {
                        float exact;
                        if (!(ok = maximum4_exact(mx * sl2 - m_sub, exact))) break;
                        if (!told) up = exact;
                    }
                    // a fresh row that sees nothing stays fresh
                    if (fresh ? up > -INFINITY : up > RESCALE_LOG2<BF16>) m = m_sub + (up - SHIFT_LOG2<BF16>);
                    const float alpha = fresh ? 1.f : ex2(m_sub - m);
                    l *= alpha;
                    if (t > t0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                        // O is at rest once PV(n - 1) is complete
                        if (!(ok = warp_wait(&ms->o_done, (n - 1) & 1, s_abort))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / GROUPS; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st16(tO + c, o);
                        }
                    }
                }
                if (both) numerators(s1);
                numerators(s0);
                // P is free once PV(n - 1) is complete
                if (n > 0) {
                    if (!(ok = warp_wait(&ms->o_done, (n - 1) & 1, s_abort))) break;
                    tc_fence_after();
                }
                if (both) tmem_st16(tP + 64, s1);
                tmem_st16(tP, s0);
                if (__builtin_expect(t + 1 == t1 && t * BN + HN * (both + 1) > it.keys, 0)) {
                    // The rows of V behind the sequence are another's or nobody's, and a NaN times a zero weight would be a
                    // NaN: they are zeroed in the tile's last piece.  (The piece's barrier is at this phase, not before: what
                    // lay there has been used by a PV that is complete.)
                    const uint32_t rv = n_v + both;
                    if (!(ok = warp_wait(&ms->v_full[rv % C::VS], (rv / C::VS) & 1, s_abort))) break;
                    uint8_t *vt = sm + C::OFF_V + (rv % C::VS) * C::PIECE;
                    for (int i = max(it.keys - t * BN - HN * both, 0) * 8 + grp * BM + r; i < HN * 8; i += GROUPS * BM)
#pragma unroll
                        for (int dh = 0; dh < D / 64; ++dh)
                            *reinterpret_cast<uint4 *>(vt + dh * HN * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                n_v += 1 + both;
                tmem_st_wait();
                tc_fence_before();
                arrive_warp(&ms->p_ready);
            }
            if (!ok) break;
            // ---- O / l, or the partial: all that does not need O first, while the last PV runs
            if (!(ok = sum4(l, l))) break;
            const int h = it.h, q_row = it.q_row;
            const bool whole = it.whole;
            arrive_warp(&ms->item_empty[n_item % NI]);
            const int64_t row = ((int64_t)q_row * a.H_q + h * a.G) + row_off;
            const int64_t prow = ((int64_t)blockIdx.x * 2 + (t0 == 0)) * BM + r;
            const bool none = l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
            // the next item's first PV overwrites O only after this thread's next P, which comes after the reads below
            if (!(ok = warp_wait(&ms->o_done, (n - 1) & 1, s_abort))) break;
            tc_fence_after();
            // A row's columns lie in one lane, so a store of them by all lanes would touch 32 lines: the warp turns its rows
            // by RS bytes each in a patch of its own in the item's Q buffer (its last S is complete), and stores eight (D =
            // 64: sixteen) rows' pieces at a time.
            constexpr int RS = D / 2, CH = RS / 16;   // bytes and 16-byte chunks of a row in the patch
            const uint32_t patch = smem_u32(sm + C::OFF_Q + (n_item & 1) * C::PIECE) + (warp - 4) * 32 * RS;
            auto place = [](int row, int chunk) { return row * RS + ((chunk ^ (CH == 4 ? (row >> 1) & 3 : (row >> 2) & 1)) << 4); };
            auto put = [&](int chunk, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(patch + place(lane, chunk)), "r"(w0), "r"(w1), "r"(w2), "r"(w3) : "memory");
            };
            // the patch to each row's place: base + RS bytes from `at` of the lane that holds the row, or nowhere if negative
            auto flush = [&](uint8_t *base, int64_t at) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int rr = i * (32 / CH) + lane / CH, ch = lane % CH;
                    const int64_t to = __shfl_sync(0xffffffffu, at, rr);
                    uint32_t w0, w1, w2, w3;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w0), "=r"(w1), "=r"(w2), "=r"(w3) : "r"(patch + place(rr, ch)) : "memory");
                    if (to >= 0) *reinterpret_cast<uint4 *>(base + to + 16 * ch) = make_uint4(w0, w1, w2, w3);
                }
                __syncwarp();
            };
            constexpr int EC = D / GROUPS;            // this thread's columns of O
            if (whole) {
#pragma unroll 1
                for (int c = 0; c < EC; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(tO + c, o);
                    tmem_ld_wait();
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = none ? 0u : pack16<BF16>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    put(c / 8, w[0], w[1], w[2], w[3]);
                    put(c / 8 + 1, w[4], w[5], w[6], w[7]);
                }
                flush(static_cast<uint8_t *>(a.out), valid ? (row * D + EC * grp) * 2 : -1);
                if (valid && grp == 0 && a.lse) a.lse[row] = none ? -INFINITY : (m + log2f(l)) * LN2;
            } else {
#pragma unroll 1
                for (int c = 0; c < EC; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(tO + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j += 4 * CH) {
#pragma unroll
                        for (int k = 0; k < CH; ++k) put(k, o[j + 4 * k], o[j + 4 * k + 1], o[j + 4 * k + 2], o[j + 4 * k + 3]);
                        flush(reinterpret_cast<uint8_t *>(a.part_o), valid ? (prow * D + EC * grp + c + j) * 4 : -1);
                    }
                }
                if (valid && grp == 0) a.part_ml[prow] = make_float2(isnan(l) ? l : m, l);   // the join passes over parts with m = -infinity
            }
            tc_fence_before();
            fence_proxy_async_smem();
            arrive_warp(&ms->q_empty[n_item & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*s_abort) {   // a wait gave up, whoever's: what is in flight ends before tensor memory is freed and the CTA exits
        volatile int never = 0;
        if (threadIdx.x == 0) atomicExch(&g_packed_status, 1);
        if (warp == 0) {
            const uint32_t n_k = ms->k_pieces, n_v = ms->v_pieces, nq = ms->q_tiles;
            for (uint32_t e = n_k > (uint32_t)C::KS ? n_k - C::KS : 0; e < n_k; ++e)
                mbar_wait(&ms->k_full[e % C::KS], (e / C::KS) & 1, &never, 200000000ull);
            for (uint32_t e = n_v > (uint32_t)C::VS ? n_v - C::VS : 0; e < n_v; ++e)
                mbar_wait(&ms->v_full[e % C::VS], (e / C::VS) & 1, &never, 200000000ull);
            for (uint32_t i = nq > 2 ? nq - 2 : 0; i < nq; ++i) mbar_wait(&ms->q_full[i & 1], (i >> 1) & 1, &never, 200000000ull);
        } else if (warp <= 2 && lane == 0) {
            umma_commit(&ms->drain[warp - 1]);
            mbar_wait(&ms->drain[warp - 1], 0, &never, 200000000ull);
        } else if (warp >= 4) {
            tmem_st_wait();
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
    }
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
    const int4 d = __ldcg(a.desc + blockIdx.x);   // first query row, tokens, kv head, partials
    if (d.w == 0) return;
    constexpr int LANES = D / 4, RPB = COMBINE_THREADS / LANES;
    const int lane = threadIdx.x % LANES;
    for (int i = threadIdx.x / LANES; i < COMBINE_ROWS; i += RPB) {
        const int r = blockIdx.y * COMBINE_ROWS + i, token = r / a.G, head = r - token * a.G;
        if (token >= d.y) continue;
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < d.w; ++p) {
            const int64_t prow = ((int64_t)(blockIdx.x + p) * 2 + (p == 0)) * BM + r;
            const float2 ml = __ldcg(a.part_ml + prow);
            if (ml.x == -INFINITY) continue;
            const float4 o = __ldcg(reinterpret_cast<const float4 *>(a.part_o + prow * D) + lane);
            const float mx = fmaxf(m, ml.x), f = m == -INFINITY ? 0.f : ex2(m - mx), w = ex2(ml.x - mx);
            m = mx;
            l = l * f + ml.y * w;
            acc.x = acc.x * f + o.x * w; acc.y = acc.y * f + o.y * w;
            acc.z = acc.z * f + o.z * w; acc.w = acc.w * f + o.w * w;
        }
        const int64_t row = (int64_t)(d.x + token) * a.H_q + d.z * a.G + head;
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
    cfg.gridDim = dim3(ctas, BM / COMBINE_ROWS);
    cfg.blockDim = dim3(COMBINE_THREADS);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, packed_combine_kernel<D, BF16>, a) != cudaSuccess) return KVC_ECUDA;
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ECUDA;
}

}  // namespace

size_t packed_scratch_bytes(int, int, int, int, int head_dim) {
    return (size_t)sm_count() * (sizeof(int4) + 2 * BM * (head_dim * sizeof(float) + sizeof(float2)));
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
    a.part_o = reinterpret_cast<float *>(a.desc + ctas);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)ctas * 2 * BM * p.D);
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)p.D);
    a.stall_ns = take_test_stall(KVC_TEST_PACKED);
    const bool bf = p.dtype == KVC_IN_BF16;
    const CUtensorMapDataType dt = bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap tq, tk, tv;
    const bool none = p.n_k == 0;   // no keys: the maps of K and V are never loaded from a row that exists
    auto map = [&](CUtensorMap *m, const void *base, int heads, int rows, int64_t ld, int box_heads, int box_rows) {
        return make_map_3d(m, dt, base, p.D, heads, rows, (uint64_t)p.D * 2, (uint64_t)ld * 2, 64, box_heads, box_rows,
                           CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!map(&tq, p.q, p.H_q, p.n_q, p.ld_q, a.G, a.tok) ||
        !map(&tk, none ? p.q : p.k, p.H_kv, none ? 1 : p.n_k, none ? p.ld_q : p.ld_k, 1, HN) ||
        !map(&tv, none ? p.q : p.v, p.H_kv, none ? 1 : p.n_k, none ? p.ld_q : p.ld_v, 1, HN))
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
