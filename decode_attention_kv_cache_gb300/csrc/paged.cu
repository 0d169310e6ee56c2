// Storing packed rows on a pool's pages, and reading them back.
//
// append: a row's values are quantised to q8_0 (blocks of 32 along head_dim: d = fp16(amax/127), codes
// round(x / (amax/127)); the arithmetic is quant.cuh's, so the bytes are kv_cache_append's) or rounded to
// fp16.  read: x = d * q in float32 (exact: 11 and 8 significant bits), rounded once to the output type.
// Both only move bytes: what bounds them is HBM, and for a few rows the latency of the dependent loads that
// find a row's page (row_start, len, the table, then the data).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace kvc {
namespace {

constexpr int THREADS = 256;

struct Pool {
    void *kq, *vq;
    uint16_t *ks, *vs;
    Geom g;
    int layer, H, D;
};

Pool pool_of(const kvc_cache &c, int layer) {
    return {c.k_q, c.v_q, static_cast<uint16_t *>(c.k_s), static_cast<uint16_t *>(c.v_s), geom_of(c.d), layer,
            c.d.n_head_kv, c.d.head_dim};
}

// One thread takes eight consecutive values of a row, of K and of V: their loads are in flight together and
// share the search for the page.  The four lanes of a q8_0 block find its amax by two shuffles, so input,
// codes and scales are all read and written in consecutive lanes' order.
template <int DT, bool Q8>
__global__ void __launch_bounds__(THREADS)
    paged_append_kernel(const void *__restrict__ k, const void *__restrict__ v, int64_t ld_k, int64_t ld_v,
                        int64_t n_units, int units_per_row, const int32_t *row_start, const PagedView pg,
                        const Pool p) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t u = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    const bool live = u < n_units;   // a multiple of four: whole blocks
    const int row = live ? (int)(u / units_per_row) : 0;
    const int e = live ? (int)(u - (int64_t)row * units_per_row) * 8 : 0;   // first value within the row
    float x[2][8] = {};
    if (live) {
        load_inputs8<DT>(k, row * ld_k + e, x[0]);
        load_inputs8<DT>(v, row * ld_v + e, x[1]);
    }
    const int slot = live ? row_slot(pg, row_start, row) : -1;
    const int head = e / p.D, c = e - head * p.D;
    const int64_t at = p.layer * p.g.c_layer + slot * p.g.c_tok + head * p.g.c_head + c;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        if constexpr (Q8) {
            uint32_t w[2];
            const uint16_t scale = q8_0_quantize_quad(x[kv], w);
            if (slot >= 0) {
                *reinterpret_cast<uint2 *>(static_cast<int8_t *>(kv ? p.vq : p.kq) + at) = make_uint2(w[0], w[1]);
                if ((c & 31) == 0)
                    (kv ? p.vs : p.ks)[p.layer * p.g.s_layer + slot * p.g.s_tok + head * p.g.s_head + (c >> 5)] = scale;
            }
        } else if (slot >= 0) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ptx::pack_half2(x[kv][2 * i], x[kv][2 * i + 1]);
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(kv ? p.vq : p.kq) + at) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(int dtype_bf16, float lo, float hi) {
    uint32_t r;
    if (dtype_bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One thread takes the values of one 16-byte load of the pool (16 codes of one block, or 8 fp16 values), of K
// and of V.
template <int DT, bool Q8>
__global__ void __launch_bounds__(THREADS)
    paged_read_kernel(void *__restrict__ k, void *__restrict__ v, int64_t n_units, int units_per_row,
                      const int32_t *row_start, const PagedView pg, const Pool p) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int N = Q8 ? 16 : 8;
    const int64_t u = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (u >= n_units) return;
    const int row = (int)(u / units_per_row);
    const int e = (int)(u - (int64_t)row * units_per_row) * N;
    const int slot = row_slot(pg, row_start, row);
    if (slot == -2) return;
    const int head = e / p.D, c = e - head * p.D;
    const int64_t at = p.layer * p.g.c_layer + slot * p.g.c_tok + head * p.g.c_head + c;
    uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    float d[2] = {0.f, 0.f};
    if (slot >= 0) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            raw[kv] = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(kv ? p.vq : p.kq) +
                                                             at * (Q8 ? 1 : 2)));
            if (Q8)
                d[kv] = __half2float(__ushort_as_half(__ldcg(
                    (kv ? p.vs : p.ks) + p.layer * p.g.s_layer + slot * p.g.s_tok + head * p.g.s_head + (c >> 5))));
        }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float x[N];
        const uint32_t w[4] = {raw[kv].x, raw[kv].y, raw[kv].z, raw[kv].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (Q8) {
#pragma unroll
                for (int b = 0; b < 4; ++b) x[4 * i + b] = (float)(int8_t)(w[i] >> (8 * b)) * d[kv];
            } else {
                x[2 * i] = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xFFFF)));
                x[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
            }
        }
        uint8_t *dst = static_cast<uint8_t *>(kv ? v : k) + u * N * (DT == KVC_IN_F32 ? 4 : 2);
        if constexpr (DT == KVC_IN_F32) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4 *>(dst + 4 * i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 8) {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = pack2(DT == KVC_IN_BF16, x[i + 2 * j], x[i + 2 * j + 1]);
                *reinterpret_cast<uint4 *>(dst + 2 * i) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

cudaLaunchConfig_t config(int64_t n_units, cudaLaunchAttribute *attr, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n_units + THREADS - 1) / THREADS));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <int DT, bool Q8>
cudaError_t append_t(const kvc_cache &c, const kvc_pages &pg, int layer, const int32_t *row_start, int n_rows,
                     const void *k, const void *v, int64_t ld_k, int64_t ld_v, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const int per_row = c.d.n_head_kv * (c.d.head_dim / 8);
    const int64_t n = (int64_t)n_rows * per_row;
    const cudaLaunchConfig_t cfg = config(n, attr, s);
    return cudaLaunchKernelEx(&cfg, paged_append_kernel<DT, Q8>, k, v, ld_k, ld_v, n, per_row, row_start,
                              paged_view(c, pg), pool_of(c, layer));
}

template <int DT, bool Q8>
cudaError_t read_t(const kvc_cache &c, const kvc_pages &pg, int layer, const int32_t *row_start, int n_rows, void *k,
                   void *v, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const int per_row = c.d.n_head_kv * (c.d.head_dim / (Q8 ? 16 : 8));
    const int64_t n = (int64_t)n_rows * per_row;
    const cudaLaunchConfig_t cfg = config(n, attr, s);
    return cudaLaunchKernelEx(&cfg, paged_read_kernel<DT, Q8>, k, v, n, per_row, row_start, paged_view(c, pg),
                              pool_of(c, layer));
}

int done(cudaError_t e) { return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? KVC_OK : KVC_ECUDA; }

}  // namespace

int launch_paged_append(const kvc_cache &c, const kvc_pages &p, int layer, const int32_t *row_start, int n_rows,
                        const void *k, const void *v, int64_t ld_k, int64_t ld_v, int dtype, cudaStream_t s) {
    const bool q8 = c.d.type == KVC_Q8_0;
    switch (dtype) {
#define KVC_CASE(DT)                                                                                       \
    case DT:                                                                                               \
        return done(q8 ? append_t<DT, true>(c, p, layer, row_start, n_rows, k, v, ld_k, ld_v, s)            \
                       : append_t<DT, false>(c, p, layer, row_start, n_rows, k, v, ld_k, ld_v, s));
        KVC_CASE(KVC_IN_F32)
        KVC_CASE(KVC_IN_BF16)
        KVC_CASE(KVC_IN_F16)
#undef KVC_CASE
        default: return KVC_EINVAL;
    }
}

int launch_paged_read(const kvc_cache &c, const kvc_pages &p, int layer, const int32_t *row_start, int n_rows, void *k,
                      void *v, int dtype, cudaStream_t s) {
    const bool q8 = c.d.type == KVC_Q8_0;
    switch (dtype) {
#define KVC_CASE(DT)                                                                        \
    case DT:                                                                                \
        return done(q8 ? read_t<DT, true>(c, p, layer, row_start, n_rows, k, v, s)            \
                       : read_t<DT, false>(c, p, layer, row_start, n_rows, k, v, s));
        KVC_CASE(KVC_IN_F32)
        KVC_CASE(KVC_IN_BF16)
        KVC_CASE(KVC_IN_F16)
#undef KVC_CASE
        default: return KVC_EINVAL;
    }
}

}  // namespace kvc
