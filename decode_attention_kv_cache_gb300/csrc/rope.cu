// Norms of queries and keys for each head and the rotation by position, in one pass; with the keys and values stored on
// a pool's pages in the same pass where asked.
//
//   y_i = x_i w_i / sqrt(mean_j x_j^2 + eps),   (a, b) -> (a cos t - b sin t, a sin t + b cos t)  for each pair,
// so that with A_i = w_i cos t, B_i = -+ w_p sin t (p the other of the pair) and r = 1 / sqrt(..)
//   out_i = r (x_i A_i + x_p B_i):
// A and B are the same for all heads of a row and are made once for it, in shared memory.  Only bytes move: what bounds it is
// HBM, and for a few rows the chain position -> angle -> table -> store.
//
// Angles.  A pair's frequency is a 64-bit fixed-point fraction f of a turn for each position, so that position times f, modulo
// 2^64, is the angle's fraction of a turn to 2^-33 whatever the position; its upper 32 bits go through sincospi.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace kvc {
namespace {

constexpr int THREADS = 128;
constexpr int BATCH = 4;   // heads whose loads a lane has in flight
constexpr int MAX_ROWS = 8;

struct Args {
    RopeArgs a;
    int lanes_log2;        // lanes of a head: eight values each, a power of two
    int rows, span;        // rows and heads that a CTA takes
    int heads;             // of a row: queries, keys, values (if stored)
    float inv_d;           // 1 / D
    // the pool, of the layer
    PagedView pg;
    const int32_t *row_start;
    uint8_t *kq, *vq;
    uint16_t *ks, *vs;
    int64_t c_tok, c_head, s_tok, s_head;
    int type;
};

template <int DT>
__device__ __forceinline__ float weight_at(const void *w, int i) {
    if (w == nullptr) return 1.f;
    if constexpr (DT == KVC_IN_F32) return __ldg(static_cast<const float *>(w) + i);
    else if constexpr (DT == KVC_IN_BF16) return __bfloat162float(__ldg(static_cast<const __nv_bfloat16 *>(w) + i));
    else return __half2float(__ldg(static_cast<const __half *>(w) + i));
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

// STORE: keys and values go to the pool, at places that the pages give, and so do the positions.
template <int DT, int STYLE, bool STORE>
__global__ void __launch_bounds__(THREADS) qk_norm_rope_kernel(const Args p) {
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ float4 table[];   // [row][queries, keys][4][chunk]: (A, B) of values 2 j, 2 j + 1 of each chunk of eight
    __shared__ int s_pos[MAX_ROWS], s_slot[MAX_ROWS];   // slot: -1 a hole, -2 a row that belongs to no sequence
    const RopeArgs &a = p.a;
    const int tid = threadIdx.x, chunks = a.D >> 3, lanes = 1 << p.lanes_log2;
    const int chunk = tid & (lanes - 1), grp = tid >> p.lanes_log2, groups = THREADS >> p.lanes_log2;
    const int row0 = blockIdx.x * p.rows, rows = min(p.rows, a.n_rows - row0);
    const int head0 = blockIdx.y * p.span, span = min(p.span, p.heads - head0), items = rows * span;
    const bool mine = chunk < chunks;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    Raw8<DT> raw[BATCH];
    auto load = [&](int base) {   // the batch's items grp + base, + groups, ...
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int item = base + i * groups + grp;
            raw[i] = Raw8<DT>{};
            if (item >= items || !mine) continue;
            const int r = item / span, h = head0 + item - r * span;
            const int64_t row = row0 + r;
            const int c = 8 * chunk;
            if (h < a.H_q) raw[i] = load_raw8<DT>(a.q, row * a.ld_q + h * a.D + c);
            else if (h < a.H_q + a.H_kv) raw[i] = load_raw8<DT>(a.k, row * a.ld_k + (h - a.H_q) * a.D + c);
            else raw[i] = load_raw8<DT>(a.v, row * a.ld_v + (h - a.H_q - a.H_kv) * a.D + c);
        }
    };
    load(0);

    // ---- where the rows are
    if constexpr (STORE) {
        const int warp = tid >> 5, lane = tid & 31;
        for (int r = warp; r < rows; r += THREADS / 32) {
            const int row = row0 + r, i = find_seq_warp(p.row_start, p.pg.n_seq, row);
            if (lane == 0) {
                const int s0 = __ldcg(p.row_start + i), s1 = __ldcg(p.row_start + i + 1), len = max(__ldcg(p.pg.len + i), 0);
                const int pos = len - (s1 - row);
                s_pos[r] = pos;
                s_slot[r] = s0 <= row && row < s1 ? page_slot(p.pg, i, pos) : -2;
            }
        }
        __syncthreads();
    }
    // ---- A and B
    for (int idx = tid; idx < rows * a.D; idx += THREADS) {
        const int r = idx / a.D, i = idx - r * a.D, n = a.n_pairs;
        float c = 1.f, s = 0.f;
        int other = i;
        if (i < 2 * n) {
            const int pair = STYLE == KVC_ROPE_HALF ? (i < n ? i : i - n) : i >> 1;
            other = STYLE == KVC_ROPE_HALF ? (i < n ? i + n : i - n) : i ^ 1;
            const long long pos = STORE ? s_pos[r] : __ldcg(a.pos + row0 + r);
            const long long t = (long long)(__ldg(a.turns + pair) * (unsigned long long)pos);
            sincospif((float)(int)(t >> 32) * 0x1p-31f, &s, &c);
            if (STYLE == KVC_ROPE_HALF ? i < n : !(i & 1)) s = -s;
        }
        float2 *at = reinterpret_cast<float2 *>(table + (r * 8 + ((i & 7) >> 1)) * chunks + (i >> 3)) + (i & 1);
        at[0] = make_float2(weight_at<DT>(a.q_weight, i) * c, weight_at<DT>(a.q_weight, other) * s);
        at[8 * chunks] = make_float2(weight_at<DT>(a.k_weight, i) * c, weight_at<DT>(a.k_weight, other) * s);
    }
    __syncthreads();

    const int n8 = a.n_pairs >> 3;   // chunks of half of a rotation in halves
    const int partner = (tid & 31 & ~(lanes - 1)) | (chunk < n8 ? chunk + n8 : chunk < 2 * n8 ? chunk - n8 : chunk);
    for (int base = 0; base < items; base += BATCH * groups) {
        if (base > 0) load(base);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int item = base + i * groups + grp;
            if (base + i * groups >= items) break;
            const bool some = item < items;
            const int r = some ? item / span : 0, h = head0 + item - r * span;
            const int kind = h < a.H_q ? 0 : h < a.H_q + a.H_kv ? 1 : 2;
            float x[8], y[8];
            widen8<DT>(raw[i], x);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
            for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if constexpr (STYLE == KVC_ROPE_HALF) {
                Raw8<DT> other;
                other.u[0] = shfl4(raw[i].u[0], partner);
                if constexpr (DT == KVC_IN_F32) other.u[1] = shfl4(raw[i].u[1], partner);
                widen8<DT>(other, y);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
            }
            if (kind < 2) {
                const float inv = (kind == 0 ? a.q_weight : a.k_weight) ? rsqrtf(fmaf(ss, p.inv_d, a.eps)) : 1.f;
                const float4 *t = table + (r * 8 + 4 * kind) * chunks + min(chunk, chunks - 1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 ab = t[j * chunks];
                    x[2 * j] = inv * fmaf(x[2 * j], ab.x, y[2 * j] * ab.y);
                    x[2 * j + 1] = inv * fmaf(x[2 * j + 1], ab.z, y[2 * j + 1] * ab.w);
                }
            }
            const Raw8<DT> out = narrow8<DT>(x);
            const int64_t row = row0 + r;
            if (kind == 0) {
                if (some && mine && (!STORE || s_slot[r] != -2)) store_raw8<DT>(a.q_out, row * a.ld_qo + h * a.D + 8 * chunk, out);
            }
            if constexpr (!STORE) {
                if (kind == 1 && some && mine) store_raw8<DT>(a.k_out, row * a.ld_ko + (h - a.H_q) * a.D + 8 * chunk, out);
            } else {
                const int slot = some && mine && kind > 0 ? s_slot[r] : -1;
                if (!__any_sync(0xffffffffu, slot >= 0)) continue;
                // as kv_paged_append stores a row of these
                widen8<DT>(out, x);
                const int head = h - a.H_q - (kind == 2 ? a.H_kv : 0), c = 8 * chunk;
                const int64_t at = slot * p.c_tok + head * p.c_head + c, sat = slot * p.s_tok + head * p.s_head + (c >> 5);
                uint8_t *codes = kind == 2 ? p.vq : p.kq;
                uint16_t *scales = kind == 2 ? p.vs : p.ks;
                if (p.type == KVC_F16) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = ptx::pack_half2(x[2 * j], x[2 * j + 1]);
                    if (slot >= 0) *reinterpret_cast<uint4 *>(codes + 2 * at) = make_uint4(w[0], w[1], w[2], w[3]);
                } else if (p.type == KVC_Q8_0) {
                    uint32_t w[2];
                    const uint16_t d = q8_0_quantize_quad(x, w);
                    if (slot >= 0) {
                        *reinterpret_cast<uint2 *>(codes + at) = make_uint2(w[0], w[1]);
                        if ((c & 31) == 0) scales[sat] = d;
                    }
                } else {
                    uint32_t w;
                    const uint16_t d = q4_0_quantize_quad(x, w);
                    if (slot >= 0) {
                        *reinterpret_cast<uint32_t *>(codes + (at >> 1)) = w;
                        if ((c & 31) == 0) scales[sat] = d;
                    }
                }
            }
        }
    }
}

template <int DT, int STYLE, bool STORE>
int launch_t(const Args &p, dim3 grid, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (size_t)p.rows * p.a.D * 2 * sizeof(float2);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<DT, STYLE, STORE>, p) != cudaSuccess) return KVC_ECUDA;
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ECUDA;
}

template <bool STORE>
int launch_all(Args p, cudaStream_t s) {
    const int chunks = p.a.D / 8;
    p.inv_d = 1.f / p.a.D;
    p.lanes_log2 = 2;
    while ((1 << p.lanes_log2) < chunks) ++p.lanes_log2;
    p.heads = p.a.H_q + p.a.H_kv * (STORE ? 2 : 1);
    const int groups = THREADS >> p.lanes_log2;
    // A CTA for every few heads of a row where there are few rows, so that all SMs take part; else whole rows, as many as make a
    // batch for every lane.
    const int64_t items = (int64_t)p.a.n_rows * p.heads;
    if (items < (int64_t)groups * BATCH * 4 * sm_count()) {
        p.rows = 1;
        p.span = groups < p.heads ? groups : p.heads;
    } else {
        const int want = (groups * BATCH + p.heads - 1) / p.heads;
        p.rows = want < MAX_ROWS ? want : MAX_ROWS;
        p.span = p.heads;
    }
    const dim3 grid((p.a.n_rows + p.rows - 1) / p.rows, (p.heads + p.span - 1) / p.span);
    switch (p.a.dtype * 2 + p.a.style) {
        case KVC_IN_F32 * 2: return launch_t<KVC_IN_F32, KVC_ROPE_HALF, STORE>(p, grid, s);
        case KVC_IN_F32 * 2 + 1: return launch_t<KVC_IN_F32, KVC_ROPE_PAIRS, STORE>(p, grid, s);
        case KVC_IN_BF16 * 2: return launch_t<KVC_IN_BF16, KVC_ROPE_HALF, STORE>(p, grid, s);
        case KVC_IN_BF16 * 2 + 1: return launch_t<KVC_IN_BF16, KVC_ROPE_PAIRS, STORE>(p, grid, s);
        case KVC_IN_F16 * 2: return launch_t<KVC_IN_F16, KVC_ROPE_HALF, STORE>(p, grid, s);
        case KVC_IN_F16 * 2 + 1: return launch_t<KVC_IN_F16, KVC_ROPE_PAIRS, STORE>(p, grid, s);
        default: return KVC_EINVAL;
    }
}

}  // namespace

int launch_rope(const RopeArgs &a, cudaStream_t s) {
    Args p = {};
    p.a = a;
    return launch_all<false>(p, s);
}

int launch_rope_append(const RopeArgs &a, const kvc_cache &c, const kvc_pages &pages, int layer, const int32_t *row_start,
                       cudaStream_t s) {
    const Geom g = geom_of(c.d);
    Args p = {};
    p.a = a;
    p.pg = paged_view(c, pages);
    p.row_start = row_start;
    p.kq = static_cast<uint8_t *>(c.k_q) + code_bytes(c.d.type, layer * g.c_layer);
    p.vq = static_cast<uint8_t *>(c.v_q) + code_bytes(c.d.type, layer * g.c_layer);
    if (has_scales(c.d.type)) {
        p.ks = static_cast<uint16_t *>(c.k_s) + layer * g.s_layer;
        p.vs = static_cast<uint16_t *>(c.v_s) + layer * g.s_layer;
    }
    p.c_tok = g.c_tok;
    p.c_head = g.c_head;
    p.s_tok = g.s_tok;
    p.s_head = g.s_head;
    p.type = c.d.type;
    return launch_all<true>(p, s);
}

}  // namespace kvc
