// Causal attention of packed prompts with grouped heads: the plain form of the kernel.
//
// Sequence s has nq query rows and nk keys; row i sees the keys j <= i + nk - nq:
//   out[i][h] = sum_j softmax_j(q[i][h] . k[j][h/G] / sqrt(D)) v[j][h/G].
// One warp per (row, query head); a lane holds D/32 dimensions and the row's running maximum and sum are kept in
// float32, one pass over the keys.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace kvc {
namespace {

template <class T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(__half &d, float x) { d = __float2half_rn(x); }
__device__ __forceinline__ void narrow(__nv_bfloat16 &d, float x) { d = __float2bfloat16_rn(x); }

template <class T, int D>
__global__ void __launch_bounds__(128) packed_kernel(const PackedArgs a, float scale) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int E = D / 32;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int row = (int)(w / a.H_q), h = (int)(w - (int64_t)row * a.H_q), kvh = h / (a.H_q / a.H_kv);
    if (row >= a.n_q) return;
    const int seq = find_seq(a.q_start, a.n_seq, row);
    if (row < __ldcg(a.q_start + seq) || row >= __ldcg(a.q_start + seq + 1)) return;
    const int k0 = max(__ldcg(a.k_start + seq), 0), k1 = min(__ldcg(a.k_start + seq + 1), a.n_k);
    const int last = k1 - (__ldcg(a.q_start + seq + 1) - row);   // the last key row this row sees
    const T *q = static_cast<const T *>(a.q) + row * a.ld_q + (int64_t)h * D;
    float x[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        x[e] = widen(q[e * 32 + lane]) * scale;
        o[e] = 0.f;
    }
    for (int j = k0; j <= last; ++j) {
        const T *k = static_cast<const T *>(a.k) + j * a.ld_k + (int64_t)kvh * D;
        const T *v = static_cast<const T *>(a.v) + j * a.ld_v + (int64_t)kvh * D;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(x[e], widen(k[e * 32 + lane]), s);
#pragma unroll
        for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        const float m_new = fmaxf(m, s), c = __expf(m - m_new), p = __expf(s - m_new);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * widen(v[e * 32 + lane]);
        m = m_new;
    }
    T *out = static_cast<T *>(a.out) + (int64_t)row * a.H_q * D + (int64_t)h * D;
#pragma unroll
    for (int e = 0; e < E; ++e) narrow(out[e * 32 + lane], l > 0.f ? o[e] / l : 0.f);
    if (a.lse && lane == 0) a.lse[(int64_t)row * a.H_q + h] = l > 0.f ? m + __logf(l) : -INFINITY;
}

template <class T, int D>
cudaError_t launch_t(const PackedArgs &a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.n_q * a.H_q + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, packed_kernel<T, D>, a, 1.f / sqrtf((float)D));
}

}  // namespace

size_t packed_scratch_bytes(int, int, int, int, int) { return 16; }

int launch_packed(const PackedArgs &a, void *, cudaStream_t s) {
    cudaError_t e;
    if (a.dtype == KVC_IN_BF16)
        e = a.D == 128 ? launch_t<__nv_bfloat16, 128>(a, s) : launch_t<__nv_bfloat16, 64>(a, s);
    else
        e = a.D == 128 ? launch_t<__half, 128>(a, s) : launch_t<__half, 64>(a, s);
    return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? KVC_OK : KVC_ECUDA;
}

}  // namespace kvc
