// What the kernels of decode_attn_paged share: the list of work and its runs, shared-memory loads, and the kernel that joins
// the partials of pairs cut by the ends of runs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace kvc {
namespace paged {

using namespace ptx;

constexpr int COMBINE_THREADS = 256;   // of a join, unless said otherwise
// A row's reference lies SHIFT_LOG2 below its greatest score, so that the numerators are 2^7 there (2^15 at most before the
// reference is raised) and fp16 holds them down to 2^-31 of it.  With the reference at the score itself those below 2^-25
// vanished from O, but not from the sum: long contexts lost them.
constexpr float SHIFT_LOG2 = 7.0f, RESCALE_LOG2 = SHIFT_LOG2 + 8.0f;
constexpr float LN2 = 0.69314718055994531f;

// What the kernels need besides the pages; a slot is a CTA (q4_0: a warp) and its run of the list.
struct Args {
    const uint16_t *ks, *vs;             // scales of the layer
    int64_t s_tok, s_head;
    const uint8_t *q;
    int64_t ld_q;                        // bytes
    void *out;
    float *lse;
    float *part_o;                       // [slot][2][G][D]
    float2 *part_ml;                     // [slot][2][G]
    int4 *desc;                          // [join]: sequence, kv head, partials (0: none), slot that begins the pair
    int H_q, H_kv, G, box, n_slots, n_q;
    int step;                            // slots from one partial of a pair to the next
    float scale_log2;
    uint64_t stall_ns;                   // test hook: > 0 makes the first consumer warp wait for what never comes
};

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
// A pair's units: its tiles of KT keys, and COST for starting and ending it.
template <int KT>
__device__ __forceinline__ int tiles_of(int keys) { return (keys + KT - 1) / KT; }
template <int KT, int COST>
__device__ __forceinline__ int units_of(int keys) { return keys > 0 ? tiles_of<KT>(keys) + COST : 0; }

// A warp's way through a run of the list: kv heads, in each the sequences, in each its units.  The
// lengths of 32 sequences are held a lane each, so that most steps load nothing.
template <int KT, int COST>
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
            const int keys = __shfl_sync(0xffffffffu, held, seq - base), all = units_of<KT, COST>(keys);
            const int x1 = (int)min((unsigned long long)all, x + left);
            p = {seq, h, max(x - COST, 0), max(x1 - COST, 0), tiles_of<KT>(keys), keys};
            left -= x1 - x;
            x = 0;
            if (++seq == pg.n_seq) { seq = 0; ++h; }
            if (p.t1 > p.t0) return true;
        }
        return false;
    }
};

// The list of W units is cut into P runs, [W c / P, W (c + 1) / P), none of them empty: one for each of n_slots CTAs (or warps), or W.
__device__ __forceinline__ unsigned long long runs_of(unsigned long long W, unsigned n_slots) {
    return min((unsigned long long)n_slots, W);
}
__device__ __forceinline__ unsigned long long run_start(unsigned long long W, unsigned n_slots, unsigned c) {
    const unsigned long long P = runs_of(W, n_slots);
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

__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
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
// Joins the partials of one pair: for each query head
// out = sum_p w_p O_p / sum_p w_p l_p, w_p = 2^(m_p - max m), the runs in a fixed order.  D / 4 threads, a group, take a
// row.  Where there are few pairs a CTA joins one head (blockIdx.y), its groups sharing the partials; else (MANY) a CTA
// joins all heads, a group each where there are few partials: 96 sequences of 64 tokens take 12.2 us, 13.5 with a CTA for
// each head, which is mostly the starting of CTAs.  The 96 sequences of 5 to 16,384 with a group for a head up to 0, 2, 8 and 32
// partials: 82, 82, 79 and 79 us, in 16 heads to a group 136, 135, 125 and 125.
constexpr int FEW_PARTS = 8;
template <int D, int DT, bool MANY, int THREADS, int B>   // B: partials that a group loads together
__device__ __forceinline__ void join_pair(const Args &a, const int4 d) {
    constexpr int LANES = D / 4, GROUPS = THREADS / LANES;
    const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    // partials first, first + step, ... of a head
    auto join = [&](int head, int first, int step, float &m, float &l, float4 &acc) {
        m = -INFINITY;
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // partial j lies with slot d.w + j step: its second place for the first (the pair begins there), else the first
        for (int j0 = first; j0 < d.z; j0 += B * step) {
            float2 ml[B];
            float4 o[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int j = j0 + b * step;
                ml[b] = make_float2(-INFINITY, 0.f);
                o[b] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < d.z) {
                    const int slot = ((d.w + j * a.step) * 2 + (j == 0)) * a.G + head;
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


// Joins blockIdx.x, blockIdx.x + gridDim.x, ... of n.
template <int D, int DT, bool MANY, int THREADS = COMBINE_THREADS, int B = 4>
__global__ void __launch_bounds__(THREADS) combine_paged_kernel(const Args a, int n) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    for (int x = blockIdx.x; x < n; x += gridDim.x) {
        const int4 d = __ldcg(a.desc + x);
        if (d.z == 0) continue;
        if (x != (int)blockIdx.x) __syncthreads();   // the join before has been read
        join_pair<D, DT, MANY, THREADS, B>(a, d);
    }
}

}  // namespace paged

// A pool of q4_0 (decode_paged_q4.cu): slots of the scratch, launch (Args as filled for every type).
int paged_q4_slots(int G);
int launch_decode_paged_q4(const kvc_cache &c, const kvc_pages &p, int layer, int dtype, const paged::Args &args, cudaStream_t s);

}  // namespace kvc
