// Norms of queries and keys for each head and the rotation by position, in one pass; with the keys and values stored on
// a pool's pages in the same pass where asked.
//
//   y_i = x_i w_i / sqrt(mean_j x_j^2 + eps),   (a, b) -> (a cos t - b sin t, a sin t + b cos t)  for each pair,
// so that with A_i = w_i cos t, B_i = -+ w_p sin t (p the other of the pair) and r = 1 / sqrt(..)
//   out_i = r (x_i A_i + x_p B_i):
// A and B are the same for all heads of a row.  A warp takes a row, or some of its heads where there are few rows: it makes
// the sines once, keeps A and B of its values in registers and goes through the heads with several loads in flight.  Only
// bytes move: HBM bounds it, and for a few rows the chain position -> angle -> store.  What else costs is instructions: where
// both of a pair lie in one lane, and two values share each multiplication (fma.f32x2), a row of 48 heads takes a warp 2,300 (issue
// slots 51% busy); heads that rotate in part, in halves, and heads of 32, 96 and the like have a kernel in which each lane
// exchanges and widens the other values as well.
//
// Measured (40 query and 8 kv heads of 128, bf16, of the rate of a copy): 10,041 rows 41.8 us (5.9 TB/s, 0.87); with keys and
// values stored, 12,711 rows on q8_0 pages 64.6 (0.77), q4_0 64.3 (0.75), f16 60.6 (0.88); 96 rows 3.6, 64 on f16 pages 4.3.  With 64
// of the 128 rotated in halves, by exchange, 52.0 (0.70), 80.6, 81.1 and 74.0.  Five heads of a lane in flight (two of those that are
// stored) and 5 CTAs per SM; with 2 heads and 6 CTAs 42.1, 67.5 (q4_0) and 63.8 (f16); with 4 and 6 44.0, 68.1 and 62.6.
//
// Angles.  A pair's frequency is a 64-bit fixed-point fraction f of a turn for each position, so that position times f, modulo
// 2^64, is the angle's fraction of a turn whatever the position; its upper 32 bits are used.  The nearest quarter of a turn is taken
// off them as integers, and what is left, an eighth of a turn at most, is rounded to float32 (2^-28 of a turn) for sincospi.  (The
// whole fraction as a float32 was off by up to 2^-26 of a turn, and sines near half a turn by as much.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kvc_internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace kvc {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int MAX_PAIRS = 128;
constexpr int NO_POOL = -1;
// Warps for an SM that a row is cut for where there are few rows.
template <int CT>
constexpr int WARPS_PER_SM = CT == NO_POOL ? 16 : 4;

struct Args {
    RopeArgs a;
    bool halves;           // a lane takes eight values of each half of a head, else eight values
    int lanes_log2;        // lanes of a head, a power of two
    int span;              // heads that a warp takes: a multiple of those that it takes at a time
    int heads;             // of a row: queries, keys, values (if stored)
    float inv_d;           // 1 / D
    // the pool, of the layer
    PagedView pg;
    const int32_t *row_start;
    uint8_t *kq, *vq;
    uint16_t *ks, *vs;
    int64_t c_tok, c_head, s_tok, s_head;
};

// Plain loads: what a kernel just before wrote is seen behind griddepcontrol.wait, and the warps of an SM share L1's copy.
template <int DT>
__device__ __forceinline__ float weight_at(const void *w, int i) {
    if constexpr (DT == KVC_IN_F32) return static_cast<const float *>(w)[i];
    else if constexpr (DT == KVC_IN_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i]);
    else return __half2float(static_cast<const __half *>(w)[i]);
}
// Eight of them; they may lie on any boundary of their type.
template <int DT>
__device__ __forceinline__ void weights8(const void *w, int i, float (&x)[8]) {
    if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {
        const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(w) + i * (DT == KVC_IN_F32 ? 4 : 2));
        Raw8<DT> r;
        r.u[0] = at[0];
        if constexpr (DT == KVC_IN_F32) r.u[1] = at[1];
        widen8<DT>(r, x);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = weight_at<DT>(w, i + j);
    }
}

// x rounded to the type, as it lies in memory.
template <int DT>
__device__ __forceinline__ Raw8<DT> narrow8(const float (&x)[8]) {
    Raw8<DT> r;
    if constexpr (DT == KVC_IN_F32) {
        r.u[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        r.u[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == KVC_IN_F16) {
                w[i] = ptx::pack_half2(x[2 * i], x[2 * i + 1]);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        r.u[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return r;
}
template <int DT>
__device__ __forceinline__ void store_raw8(void *base, int64_t idx, const Raw8<DT> &r) {
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(base) + idx * (DT == KVC_IN_F32 ? 4 : 2));
    p[0] = r.u[0];
    if constexpr (DT == KVC_IN_F32) p[1] = r.u[1];
}
__device__ __forceinline__ uint4 shfl4(const uint4 &u, int lane) {
    return make_uint4(__shfl_sync(0xffffffffu, u.x, lane), __shfl_sync(0xffffffffu, u.y, lane),
                      __shfl_sync(0xffffffffu, u.z, lane), __shfl_sync(0xffffffffu, u.w, lane));
}

// The row's position and place in the pool (-1: a hole); false: a row that belongs to no sequence.
template <int CT>
__device__ __forceinline__ bool place_of(const Args &p, int row, int &pos, int &slot) {
    slot = -1;
    if constexpr (CT == NO_POOL) {
        pos = __ldcg(p.a.pos + row);
    } else {
        const int i = find_seq_warp(p.row_start, p.pg.n_seq, row);
        const int s0 = __ldcg(p.row_start + i), s1 = __ldcg(p.row_start + i + 1), len = max(__ldcg(p.pg.len + i), 0);
        if (row < s0 || row >= s1) return false;
        pos = len - (s1 - row);
        slot = page_slot(p.pg, i, pos);
    }
    return true;
}

// (cosine, sine) of each of the row's pairs; those behind the rotation do not turn.
__device__ __forceinline__ void turn(const RopeArgs &a, int pos, int lane, float2 *turned) {
    for (int pair = lane; pair < a.D >> 1; pair += 32) {
        float s = 0.f, c = 1.f;
        if (pair < a.n_pairs) {
            const unsigned t = (unsigned)((a.turns[pair] * (unsigned long long)(long long)pos) >> 32);
            const unsigned quarter = (t + 0x20000000u) >> 30;
            float y, x;
            sincospif((float)(int)(t - (quarter << 30)) * 0x1p-31f, &y, &x);
            c = quarter & 1 ? y : x;
            s = quarter & 1 ? x : y;
            if (quarter == 1 || quarter == 2) c = -c;
            if (quarter >= 2) s = -s;
        }
        turned[pair] = make_float2(c, s);
    }
    __syncwarp();
}

// Eight values of a key (or a value), stored as kv_paged_append does; all lanes of a block's four call.
template <int DT, int CT>
__device__ __forceinline__ void store_kv(const Args &p, bool value, bool some, int slot, int h, int chunk, const float (&x)[8]) {
    const int e = 8 * chunk;
    const int64_t at = slot * p.c_tok + h * p.c_head + e, sat = slot * p.s_tok + h * p.s_head + (e >> 5);
    uint8_t *codes = value ? p.vq : p.kq;
    uint16_t *scales = value ? p.vs : p.ks;
    if constexpr (CT == KVC_F16) {
        uint32_t w4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w4[j] = ptx::pack_half2(x[2 * j], x[2 * j + 1]);
        if (some) *reinterpret_cast<uint4 *>(codes + 2 * at) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
    } else if constexpr (CT == KVC_Q8_0) {
        uint32_t w2[2];
        const uint16_t d = q8_0_quantize_quad<DT>(x, w2);
        if (some) {
            *reinterpret_cast<uint2 *>(codes + at) = make_uint2(w2[0], w2[1]);
            if ((e & 31) == 0) scales[sat] = d;
        }
    } else {
        uint32_t w1;
        const uint16_t d = q4_0_quantize_quad<DT>(x, w1);
        if (some) {
            *reinterpret_cast<uint32_t *>(codes + (at >> 1)) = w1;
            if ((e & 31) == 0) scales[sat] = d;
        }
    }
}

// What both kernels begin with.  CT: the pool's type, or NO_POOL.  With a pool keys and values go there, to places that the
// pages give, and so do the positions.
#define KVC_ROPE_BEGIN                                                             \
    asm volatile("griddepcontrol.launch_dependents;");                             \
    constexpr bool STORE = CT != NO_POOL;                                          \
    __shared__ float2 turned_all[WARPS][MAX_PAIRS];                                \
    const RopeArgs &a = p.a;                                                       \
    const int lane = threadIdx.x & 31, row = blockIdx.x * WARPS + (threadIdx.x >> 5); \
    float2 *turned = turned_all[threadIdx.x >> 5];                                 \
    if (row >= a.n_rows) return;                                                   \
    const int h0 = blockIdx.y * p.span, h1 = min(h0 + p.span, p.heads);            \
    asm volatile("griddepcontrol.wait;" ::: "memory");                             \
    int pos, slot;                                                                 \
    if (!place_of<CT>(p, row, pos, slot)) return;                                  \
    turn(a, pos, lane, turned);

// Heads of 64, 128 or 256 that rotate whole or not at all, or in pairs of neighbours: a lane takes eight values of a head's
// first half and the eight half a head behind them, so that both of a pair lie in one lane.
template <int DT, int STYLE, int CT>
__global__ void __launch_bounds__(THREADS, CT != NO_POOL && DT == KVC_IN_F32 ? 4 : 5) qk_norm_rope_halves_kernel(const Args p) {
    KVC_ROPE_BEGIN
    const int lanes = 1 << p.lanes_log2, together = 32 >> p.lanes_log2;
    const int chunk = lane & (lanes - 1), grp = lane >> p.lanes_log2;
    // Heads [first, last) of one kind: queries (0), keys (1), values (2).
    auto heads_of = [&](auto kind_tag, int first, int last) {
        constexpr int KIND = decltype(kind_tag)::value;
        constexpr int BATCH = DT == KVC_IN_F32 || (STORE && KIND > 0) ? 2 : 5;   // heads of a lane in flight
        if (first >= last) return;
        uint64_t A[2][4], B[2][4];   // of both halves, two values each
        const void *w = KIND == 0 ? a.q_weight : a.k_weight;
        const bool normed = KIND < 2 && w != nullptr;
        const void *src = KIND == 0 ? a.q : KIND == 1 ? a.k : a.v;
        const int64_t src0 = row * (KIND == 0 ? a.ld_q : KIND == 1 ? a.ld_k : a.ld_v) + 8 * chunk;
        for (int base = first; base < last; base += BATCH * together) {
            Raw8<DT> raw[BATCH][2];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int h = base + i * together + grp;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    raw[i][u] = Raw8<DT>{};
                    if (h < last) raw[i][u] = load_raw8<DT>(src, src0 + h * a.D + u * 8 * lanes);
                }
            }
            if (KIND < 2 && base == first) {
                float wt[2][8] = {{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
                if (normed) {
                    weights8<DT>(w, chunk * 8, wt[0]);
                    weights8<DT>(w, (chunk + lanes) * 8, wt[1]);
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int i = (chunk + u * lanes) * 8 + j;
                        const float2 c0 = turned[STYLE == KVC_ROPE_PAIRS ? i >> 1 : chunk * 8 + j];
                        const float2 c1 = STYLE == KVC_ROPE_PAIRS ? c0 : turned[chunk * 8 + j + 1];
                        A[u][j >> 1] = ptx::f2_pack(wt[u][j] * c0.x, wt[u][j + 1] * c1.x);
                        B[u][j >> 1] = STYLE == KVC_ROPE_PAIRS ? ptx::f2_pack(-wt[u][j + 1] * c0.y, wt[u][j] * c0.y)
                                       : u == 0                ? ptx::f2_pack(-wt[1][j] * c0.y, -wt[1][j + 1] * c1.y)
                                                               : ptx::f2_pack(wt[0][j] * c0.y, wt[0][j + 1] * c1.y);
                    }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (base + i * together >= last) break;
                const int h = base + i * together + grp;
                const bool some = h < last;
                float x[2][8];
                widen8<DT>(raw[i][0], x[0]);
                widen8<DT>(raw[i][1], x[1]);
                if constexpr (KIND < 2) {
                    uint64_t x2[2][4];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) x2[u][j] = ptx::f2_pack(x[u][2 * j], x[u][2 * j + 1]);
                    float inv = 1.f;
                    if (normed) {
                        uint64_t s2 = ptx::f2_mul(x2[0][0], x2[0][0]), t2 = ptx::f2_mul(x2[1][0], x2[1][0]);
#pragma unroll
                        for (int j = 1; j < 4; ++j) {
                            s2 = ptx::f2_fma(x2[0][j], x2[0][j], s2);
                            t2 = ptx::f2_fma(x2[1][j], x2[1][j], t2);
                        }
                        float s0, s1;
                        ptx::f2_unpack(ptx::f2_add(s2, t2), s0, s1);
                        float ss = s0 + s1;
                        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
                        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
                        if (lanes >= 8) ss += __shfl_xor_sync(0xffffffffu, ss, 4);
                        if (lanes == 16) ss += __shfl_xor_sync(0xffffffffu, ss, 8);
                        inv = rsqrtf(fmaf(ss, p.inv_d, a.eps));
                    }
                    const uint64_t inv2 = ptx::f2_pack(inv, inv);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t y2 = STYLE == KVC_ROPE_HALF ? x2[u ^ 1][j] : ptx::f2_pack(x[u][2 * j + 1], x[u][2 * j]);
                            const uint64_t o = ptx::f2_mul(inv2, ptx::f2_fma(x2[u][j], A[u][j], ptx::f2_mul(y2, B[u][j])));
                            ptx::f2_unpack(o, x[u][2 * j], x[u][2 * j + 1]);
                        }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = chunk + u * lanes;
                    if constexpr (KIND == 2) {
                        store_kv<DT, CT>(p, true, some, slot, h, c, x[u]);
                    } else {
                        const Raw8<DT> out = narrow8<DT>(x[u]);
                        if constexpr (KIND == 0) {
                            if (some) store_raw8<DT>(a.q_out, row * a.ld_qo + h * a.D + 8 * c, out);
                        } else if constexpr (!STORE) {
                            if (some) store_raw8<DT>(a.k_out, row * a.ld_ko + h * a.D + 8 * c, out);
                        } else {
                            widen8<DT>(out, x[u]);
                            store_kv<DT, CT>(p, false, some, slot, h, c, x[u]);
                        }
                    }
                }
            }
        }
    };
    const int h_k = a.H_q, h_v = a.H_q + a.H_kv;
    heads_of(std::integral_constant<int, 0>{}, h0, min(h1, h_k));
    if (!STORE || slot >= 0) {
        heads_of(std::integral_constant<int, 1>{}, max(h0, h_k) - h_k, min(h1, h_v) - h_k);
        if constexpr (STORE) heads_of(std::integral_constant<int, 2>{}, max(h0, h_v) - h_v, h1 - h_v);
    }
}

// Heads of any multiple of 32 that rotate in part: a lane takes eight values, and gets the other eight of its pairs from
// another lane.
template <int DT, int STYLE, int CT>
__global__ void __launch_bounds__(THREADS) qk_norm_rope_kernel(const Args p) {
    KVC_ROPE_BEGIN
    const int lanes = 1 << p.lanes_log2, together = 32 >> p.lanes_log2;   // heads at a time
    const int chunks = a.D >> 3, chunk = lane & (lanes - 1), grp = lane >> p.lanes_log2;
    const bool mine = chunk < chunks;
    const int own_chunk = min(chunk, chunks - 1);
    float c[8], s[8];   // of this lane's values; s with the sign of out_i's other
    const int n8 = a.n_pairs >> 3;   // chunks of half of a rotation in halves
    const int other_chunk = STYLE == KVC_ROPE_PAIRS ? own_chunk
                            : chunk < n8            ? chunk + n8
                            : chunk < 2 * n8        ? chunk - n8
                                                    : own_chunk;
    const int partner = (lane & ~(lanes - 1)) | (chunk < 2 * n8 ? other_chunk : chunk);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = own_chunk * 8 + j, n = a.n_pairs;
        c[j] = 1.f;
        s[j] = 0.f;
        if (i < 2 * n) {
            const float2 cs = turned[STYLE == KVC_ROPE_PAIRS ? i >> 1 : i < n ? i : i - n];
            c[j] = cs.x;
            s[j] = (STYLE == KVC_ROPE_PAIRS ? (j & 1) == 0 : i < n) ? -cs.y : cs.y;
        }
    }

    // Heads [first, last) of one kind: queries (0), keys (1), values (2).
    auto heads_of = [&](auto kind_tag, int first, int last) {
        constexpr int KIND = decltype(kind_tag)::value;
        constexpr int BATCH = KIND == 0 || !STORE ? (DT == KVC_IN_F32 ? 4 : 6) : 4;   // loads of a lane in flight
        if (first >= last) return;
        float A[8], B[8];
        const void *w = KIND == 0 ? a.q_weight : a.k_weight;
        const bool normed = KIND < 2 && w != nullptr;
        const void *src = KIND == 0 ? a.q : KIND == 1 ? a.k : a.v;
        const int64_t src0 = row * (KIND == 0 ? a.ld_q : KIND == 1 ? a.ld_k : a.ld_v) + 8 * own_chunk;
        for (int base = first; base < last; base += BATCH * together) {
            Raw8<DT> raw[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int h = base + i * together + grp;
                raw[i] = Raw8<DT>{};
                if (h < last && mine) raw[i] = load_raw8<DT>(src, src0 + h * a.D);
            }
            if (KIND < 2 && base == first) {
                if (normed) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {   // weights may lie on any boundary of their type
                        A[j] = weight_at<DT>(w, own_chunk * 8 + j) * c[j];
                        B[j] = weight_at<DT>(w, other_chunk * 8 + (STYLE == KVC_ROPE_PAIRS ? j ^ 1 : j)) * s[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) { A[j] = c[j]; B[j] = s[j]; }
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (base + i * together >= last) break;
                const int h = base + i * together + grp;
                const bool some = h < last && mine;
                float x[8];
                widen8<DT>(raw[i], x);
                Raw8<DT> out = raw[i];
                if constexpr (KIND < 2) {
                    float y[8];
                    if constexpr (STYLE == KVC_ROPE_HALF) {
                        Raw8<DT> other;
                        other.u[0] = shfl4(raw[i].u[0], partner);
                        if constexpr (DT == KVC_IN_F32) other.u[1] = shfl4(raw[i].u[1], partner);
                        widen8<DT>(other, y);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
                    }
                    float inv = 1.f;
                    if (normed) {
                        float ss = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
                        for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                        inv = rsqrtf(fmaf(ss, p.inv_d, a.eps));
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = inv * fmaf(x[j], A[j], y[j] * B[j]);
                    out = narrow8<DT>(x);
                }
                if constexpr (KIND == 0) {
                    if (some) store_raw8<DT>(a.q_out, row * a.ld_qo + h * a.D + 8 * chunk, out);
                } else if constexpr (!STORE) {
                    if (some) store_raw8<DT>(a.k_out, row * a.ld_ko + h * a.D + 8 * chunk, out);
                } else {
                    if constexpr (KIND == 1) widen8<DT>(out, x);
                    store_kv<DT, CT>(p, KIND == 2, some, slot, h, chunk, x);
                }
            }
        }
    };
    const int h_k = a.H_q, h_v = a.H_q + a.H_kv;
    heads_of(std::integral_constant<int, 0>{}, h0, min(h1, h_k));
    if (!STORE || slot >= 0) {
        heads_of(std::integral_constant<int, 1>{}, max(h0, h_k) - h_k, min(h1, h_v) - h_k);
        if constexpr (STORE) heads_of(std::integral_constant<int, 2>{}, max(h0, h_v) - h_v, h1 - h_v);
    }
}

#undef KVC_ROPE_BEGIN

template <int DT, int STYLE, int CT>
int launch_t(const Args &p, dim3 grid, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, p.halves ? qk_norm_rope_halves_kernel<DT, STYLE, CT> : qk_norm_rope_kernel<DT, STYLE, CT>, p) != cudaSuccess) return KVC_ECUDA;
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ECUDA;
}

template <int CT>
int launch_all(Args p, cudaStream_t s) {
    const int chunks = p.a.D / 8;
    p.inv_d = 1.f / p.a.D;
    p.halves = (chunks & (chunks - 1)) == 0 && chunks >= 8 &&
               (p.a.style == KVC_ROPE_PAIRS || p.a.n_pairs == 0 || p.a.n_pairs == p.a.D / 2);
    p.lanes_log2 = 2;
    while ((1 << p.lanes_log2) < (p.halves ? chunks / 2 : chunks)) ++p.lanes_log2;
    p.heads = p.a.H_q + p.a.H_kv * (CT != NO_POOL ? 2 : 1);
    // Whole rows for a warp where there are enough of them to keep the SMs busy; else as many warps for a row as that takes.
    const int together = 32 >> p.lanes_log2, times = (p.heads + together - 1) / together;
    const int want = (int)(((int64_t)WARPS_PER_SM<CT> * sm_count() + p.a.n_rows - 1) / p.a.n_rows), parts = want < times ? want : times;
    p.span = (times + parts - 1) / parts * together;
    const dim3 grid((unsigned)(((int64_t)p.a.n_rows + WARPS - 1) / WARPS), (p.heads + p.span - 1) / p.span);
    switch (p.a.dtype * 2 + p.a.style) {
        case KVC_IN_F32 * 2: return launch_t<KVC_IN_F32, KVC_ROPE_HALF, CT>(p, grid, s);
        case KVC_IN_F32 * 2 + 1: return launch_t<KVC_IN_F32, KVC_ROPE_PAIRS, CT>(p, grid, s);
        case KVC_IN_BF16 * 2: return launch_t<KVC_IN_BF16, KVC_ROPE_HALF, CT>(p, grid, s);
        case KVC_IN_BF16 * 2 + 1: return launch_t<KVC_IN_BF16, KVC_ROPE_PAIRS, CT>(p, grid, s);
        case KVC_IN_F16 * 2: return launch_t<KVC_IN_F16, KVC_ROPE_HALF, CT>(p, grid, s);
        case KVC_IN_F16 * 2 + 1: return launch_t<KVC_IN_F16, KVC_ROPE_PAIRS, CT>(p, grid, s);
        default: return KVC_EINVAL;
    }
}

}  // namespace
}  // namespace kvc
