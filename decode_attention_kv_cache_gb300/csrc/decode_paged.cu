// Attention of one new token for each sequence over a paged pool: the plain form of the kernel.
//
//   out[i][h] = sum_{j < len[i]} softmax_j(q[i][h] . khat[j][h/G] / sqrt(D)) vhat[j][h/G]
//
// One CTA per (sequence, query head).  Its four warps take every fourth key; a lane holds D/32 dimensions.
// Each warp keeps a running maximum and sum of its keys in float32 (one pass over the data), and the four are
// joined in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace kvc {
namespace {

struct Args {
    const void *kq, *vq;
    const uint16_t *ks, *vs;
    Geom g;
    int layer, H_q, G;
    const void *q;
    int64_t ld_q;
    void *out;
    float *lse;
    float scale;
};

template <int DT>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if constexpr (DT == KVC_IN_F32) return static_cast<const float *>(p)[i];
    else if constexpr (DT == KVC_IN_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    else return __half2float(static_cast<const __half *>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store1(void *p, int64_t i, float x) {
    if constexpr (DT == KVC_IN_F32) static_cast<float *>(p)[i] = x;
    else if constexpr (DT == KVC_IN_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    else static_cast<__half *>(p)[i] = __float2half_rn(x);
}

template <int D, bool Q8, int DT>
__global__ void __launch_bounds__(128) decode_paged_kernel(const PagedView pg, const Args a) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int E = D / 32;
    const int seq = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = max(pg.len[seq], 0), kvh = h / a.G;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = load1<DT>(a.q, seq * a.ld_q + (int64_t)h * D + e * 32 + lane) * a.scale;
        o[e] = 0.f;
    }
    auto value = [&](bool is_v, int slot, int e) -> float {
        const int64_t at = a.layer * a.g.c_layer + slot * a.g.c_tok + kvh * a.g.c_head + e * 32 + lane;
        if constexpr (Q8) {
            const uint16_t d = (is_v ? a.vs : a.ks)[a.layer * a.g.s_layer + slot * a.g.s_tok + kvh * a.g.s_head + e];
            return (float)static_cast<const int8_t *>(is_v ? a.vq : a.kq)[at] * __half2float(__ushort_as_half(d));
        } else {
            return __half2float(static_cast<const __half *>(is_v ? a.vq : a.kq)[at]);
        }
    };
    for (int j = warp; j < len; j += 4) {
        const int slot = page_slot(pg, seq, j);
        if (slot < 0) continue;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], value(false, slot, e), s);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float m_new = fmaxf(m, s), c = __expf(m - m_new), p = __expf(s - m_new);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * value(true, slot, e);
        m = m_new;
    }
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][e * 32 + lane] = o[e];
    if (lane == 0) { sm_m[warp] = m; sm_l[warp] = l; }
    __syncthreads();
    const float M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    float L = 0.f, acc = 0.f;
    if (M > -INFINITY) {
        for (int w = 0; w < 4; ++w) {
            const float c = __expf(sm_m[w] - M);
            L += c * sm_l[w];
            if (threadIdx.x < D) acc += c * sm_o[w][threadIdx.x];
        }
    }
    if (threadIdx.x < D) store1<DT>(a.out, ((int64_t)seq * a.H_q + h) * D + threadIdx.x, L > 0.f ? acc / L : 0.f);
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)seq * a.H_q + h] = M > -INFINITY ? M + __logf(L) : -INFINITY;
}

template <int D, bool Q8, int DT>
cudaError_t launch_t(const PagedView &pg, const Args &a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pg.n_seq, a.H_q);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_paged_kernel<D, Q8, DT>, pg, a);
}

template <int D, bool Q8>
cudaError_t launch_dt(int dtype, const PagedView &pg, const Args &a, cudaStream_t s) {
    switch (dtype) {
        case KVC_IN_F32: return launch_t<D, Q8, KVC_IN_F32>(pg, a, s);
        case KVC_IN_BF16: return launch_t<D, Q8, KVC_IN_BF16>(pg, a, s);
        default: return launch_t<D, Q8, KVC_IN_F16>(pg, a, s);
    }
}

}  // namespace

size_t paged_scratch_bytes(const kvc_desc &, int, int) { return 16; }

int launch_decode_paged(const kvc_cache &c, const kvc_pages &p, int layer, const void *q, int64_t ld_q, int dtype,
                        int n_head_q, void *out, float *lse, void *, cudaStream_t s) {
    Args a;
    a.kq = c.k_q;
    a.vq = c.v_q;
    a.ks = static_cast<const uint16_t *>(c.k_s);
    a.vs = static_cast<const uint16_t *>(c.v_s);
    a.g = geom_of(c.d);
    a.layer = layer;
    a.H_q = n_head_q;
    a.G = n_head_q / c.d.n_head_kv;
    a.q = q;
    a.ld_q = ld_q;
    a.out = out;
    a.lse = lse;
    a.scale = 1.f / sqrtf((float)c.d.head_dim);
    const PagedView pg = paged_view(c, p);
    const bool q8 = c.d.type == KVC_Q8_0;
    cudaError_t e;
    if (c.d.head_dim == 128) e = q8 ? launch_dt<128, true>(dtype, pg, a, s) : launch_dt<128, false>(dtype, pg, a, s);
    else e = q8 ? launch_dt<64, true>(dtype, pg, a, s) : launch_dt<64, false>(dtype, pg, a, s);
    return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? KVC_OK : KVC_ECUDA;
}

}  // namespace kvc
