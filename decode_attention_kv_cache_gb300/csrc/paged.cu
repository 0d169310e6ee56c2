// Storing packed rows on a pool's pages, and reading them back.
//
// append: a row's values are quantised to q8_0 (blocks of 32 along head_dim: d = fp16(amax/127), codes
// round(x / (amax/127)); the arithmetic is quant.cuh's, so the bytes are kv_cache_append's) or rounded to
// fp16.  read: x = d * q in float32 (exact: 11 and 8 significant bits), rounded once to the output type.
// Both only move bytes: what bounds them is HBM, and for a few rows the latency of the dependent loads that
// find a row's page (row_start, len, the table, then the data).  What bounds the q8_0 append of many rows is neither:
// the quantiser's own arithmetic, about 200 instructions for eight values.
//
// Measured (8 kv heads of 128, of the rate of a copy): 19,300 fp16 rows into an f16 cache 27.6 us (5.7 TB/s, 0.85);
// 21,100 bf16 rows into a q8_0 cache 42.1 us (3.1 TB/s, 0.46; from float32 4.5 TB/s); 58,300 positions of a q8_0 cache
// read into bf16 56.7 us (6.5 TB/s, 0.95) and of an f16 cache 71.6 us (6.7 TB/s, 0.98); eight rows appended 2.0 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace kvc {
namespace {

// Threads of a CTA, which waits for its look-ups as one: 256, 128 and 64 take 43.4, 42.1 and 42.6 us for the q8_0 append
// above (54, 49 and 49 from float32), 56.6, 56.8 and 63.7 for the q8_0 read.
constexpr int THREADS = 128;
// Units that a thread takes where there are many.  Measured at the sizes above, with 1, 2 and 4 of them: a q8_0 append
// 48.0, 42.1 and 42.6 us, an f16 append 27.7, 27.8 and 28.6; a read of a q8_0 cache, whose one load makes two stores'
// worth of values, 56.7, 57.2 and 62.7; of an f16 cache 76.8, 71.6 and 71.8.
constexpr int APPEND_PASSES = 2;
template <bool Q8>
constexpr int READ_PASSES = Q8 ? 1 : 2;

// n / d for 32-bit n by a multiplication: floor(n (2^64 / d + 1) / 2^64), where the part that is too much,
// n / 2^64, is below the 1/d that would be needed to reach the next integer.
struct Div {
    unsigned long long m;
    __device__ __forceinline__ int operator()(int n) const { return (int)__umul64hi((unsigned long long)(unsigned)n, m); }
};
Div div_of(int d) { return {~0ull / d + 1}; }   // a row has two units or more, and so has a head

struct Pool {
    void *kq, *vq;             // of the layer
    uint16_t *ks, *vs;
    int64_t c_tok, c_head, s_tok, s_head;
    Div per_row, per_head;     // units
    int units_per_row, units_per_head;
};

Pool pool_of(const kvc_cache &c, int layer, int values_per_unit) {
    const Geom g = geom_of(c.d);
    const int esz = c.d.type == KVC_Q8_0 ? 1 : 2, per_head = c.d.head_dim / values_per_unit, per_row = c.d.n_head_kv * per_head;
    const int64_t at = layer * g.c_layer * esz, sat = c.d.type == KVC_Q8_0 ? layer * g.s_layer : 0;
    return {static_cast<uint8_t *>(c.k_q) + at, static_cast<uint8_t *>(c.v_q) + at, static_cast<uint16_t *>(c.k_s) + sat,
            static_cast<uint16_t *>(c.v_s) + sat, g.c_tok, g.c_head, g.s_tok, g.s_head, div_of(per_row),
            div_of(per_head), per_row, per_head};
}

// A CTA takes THREADS * PASSES consecutive units of the packed rows (a unit: the values of one load, of K and
// of V).  The pool positions of its rows are found once, one row per thread, into shared memory.
struct Span {
    int row0;      // the CTA's first row
    int rem;       // its first unit, counted from that row's first
    int rows;      // rows that it touches
};

__device__ __forceinline__ Span span_of(int64_t n_units, int units_per_row, int units_per_cta) {
    const int64_t u0 = (int64_t)blockIdx.x * units_per_cta;
    Span s;
    s.row0 = (int)(u0 / units_per_row);
    s.rem = (int)(u0 - (int64_t)s.row0 * units_per_row);
    const int n = (int)min((int64_t)units_per_cta, n_units - u0);
    s.rows = (s.rem + n - 1) / units_per_row + 1;
    return s;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (DT == KVC_IN_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// eight 32-bit words to global memory: in one access where the address is a multiple of 32 (WIDE)
template <bool WIDE>
__device__ __forceinline__ void store8(void *dst, const uint32_t (&w)[8]) {
    if (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// One thread takes eight consecutive values of a row, of K and of V, PASSES times; all of its loads are in flight
// before the first value is used, and the look-ups overlap them.  The four lanes of a q8_0 block find its amax by
// two shuffles, so input, codes and scales are all read and written in consecutive lanes' order.
template <int DT, bool Q8, int PASSES>
__global__ void __launch_bounds__(THREADS)
    paged_append_kernel(const void *__restrict__ k, const void *__restrict__ v, int64_t ld_k, int64_t ld_v,
                        int64_t n_units, const int32_t *row_start, const PagedView pg, const Pool p) {
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ int slots[THREADS * PASSES / 4 + 1];   // a row has four units or more
    const Span sp = span_of(n_units, p.units_per_row, THREADS * PASSES);
    const int64_t left = n_units - (int64_t)blockIdx.x * (THREADS * PASSES);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Raw8<DT> raw[PASSES][2];
    int r[PASSES], e[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int u = i * THREADS + threadIdx.x;
        r[i] = p.per_row(sp.rem + u);
        e[i] = sp.rem + u - r[i] * p.units_per_row;
        if (u >= left) r[i] = -1;   // a multiple of four units: whole blocks
        if (r[i] >= 0) {
            raw[i][0] = load_raw8<DT>(k, (sp.row0 + r[i]) * ld_k + e[i] * 8);
            raw[i][1] = load_raw8<DT>(v, (sp.row0 + r[i]) * ld_v + e[i] * 8);
        } else {
            raw[i][0] = raw[i][1] = Raw8<DT>{};
        }
    }
    row_slots(pg, row_start, sp.row0, sp.rows, slots);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int slot = r[i] >= 0 ? slots[r[i]] : -1;
        const int head = p.per_head(e[i]), c = (e[i] - head * p.units_per_head) * 8;
        const int64_t at = slot * p.c_tok + head * p.c_head + c;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            float x[8];
            widen8<DT>(raw[i][kv], x);
            if constexpr (Q8) {
                uint32_t w[2];
                const uint16_t scale = q8_0_quantize_quad(x, w);
                if (slot >= 0) {
                    *reinterpret_cast<uint2 *>(static_cast<int8_t *>(kv ? p.vq : p.kq) + at) = make_uint2(w[0], w[1]);
                    if ((c & 31) == 0)
                        (kv ? p.vs : p.ks)[slot * p.s_tok + head * p.s_head + (c >> 5)] = scale;
                }
            } else if (slot >= 0) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = ptx::pack_half2(x[2 * j], x[2 * j + 1]);
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(kv ? p.vq : p.kq) + at) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// One thread takes the values of one 16-byte load of the pool (16 codes of one block, or 8 fp16 values), of K
// and of V, PASSES times, all loads in flight together.  32-byte stores where the outputs allow them.
template <int DT, bool Q8, int PASSES, bool WIDE>
__global__ void __launch_bounds__(THREADS)
    paged_read_kernel(void *__restrict__ k, void *__restrict__ v, int64_t n_units, const int32_t *row_start,
                      const PagedView pg, const Pool p) {
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int N = Q8 ? 16 : 8;
    __shared__ int slots[THREADS * PASSES / 2 + 1];   // a row has two units or more
    const Span sp = span_of(n_units, p.units_per_row, THREADS * PASSES);
    const int64_t u0 = (int64_t)blockIdx.x * (THREADS * PASSES), left = n_units - u0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    row_slots(pg, row_start, sp.row0, sp.rows, slots);
    __syncthreads();
    uint4 raw[PASSES][2];
    uint16_t d[PASSES][2];
    int slot[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int u = i * THREADS + threadIdx.x, r = p.per_row(sp.rem + u), e = sp.rem + u - r * p.units_per_row;
        const int head = p.per_head(e), c = (e - head * p.units_per_head) * N;
        slot[i] = u < left ? slots[r] : -2;
        raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
        d[i][0] = d[i][1] = 0;
        if (slot[i] < 0) continue;
        const int64_t at = slot[i] * p.c_tok + head * p.c_head + c;
        const int64_t sat = slot[i] * p.s_tok + head * p.s_head + (c >> 5);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            raw[i][kv] = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(kv ? p.vq : p.kq) +
                                                                at * (Q8 ? 1 : 2)));
            if (Q8) d[i][kv] = __ldcg((kv ? p.vs : p.ks) + sat);
        }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        if (slot[i] == -2) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            float x[N];
            const uint32_t w[4] = {raw[i][kv].x, raw[i][kv].y, raw[i][kv].z, raw[i][kv].w};
            const float s = Q8 ? __half2float(__ushort_as_half(d[i][kv])) : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (Q8) {
                    // a code plus 128 in the low bits of 2^23 is the float 2^23 + 128 + code, exactly
                    const uint32_t u = w[j] ^ 0x80808080u;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        x[4 * j + b] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540 + b)) - 8388736.f) * s;
                } else {
                    x[2 * j] = __half2float(__ushort_as_half((unsigned short)(w[j] & 0xFFFF)));
                    x[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(w[j] >> 16)));
                }
            }
            const int64_t u = u0 + i * THREADS + threadIdx.x;
            uint8_t *dst = static_cast<uint8_t *>(kv ? v : k) + u * N * (DT == KVC_IN_F32 ? 4 : 2);
            if constexpr (DT == KVC_IN_F32) {
#pragma unroll
                for (int j = 0; j < N; j += 8) {
                    uint32_t o[8];
#pragma unroll
                    for (int b = 0; b < 8; ++b) o[b] = __float_as_uint(x[j + b]);
                    store8<WIDE>(dst + 4 * j, o);
                }
            } else if constexpr (Q8) {
                uint32_t o[8];
#pragma unroll
                for (int b = 0; b < 8; ++b) o[b] = pack2<DT>(x[2 * b], x[2 * b + 1]);
                store8<WIDE>(dst, o);
            } else {
                *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]),
                                                             pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
            }
        }
    }
}

cudaLaunchConfig_t config(int64_t n_units, int units_per_cta, cudaLaunchAttribute *attr, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n_units + units_per_cta - 1) / units_per_cta));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Several passes only where there are enough units to keep every SM busy with several CTAs of that many: eight rows
// take 2.0 us with one and 2.25 with two.
bool many(int64_t n_units, int passes) { return n_units >= (int64_t)THREADS * passes * 8 * sm_count(); }

template <int DT, bool Q8, int PASSES>
cudaError_t append_p(const kvc_cache &c, const kvc_pages &pg, int layer, const int32_t *row_start, int64_t n,
                     const void *k, const void *v, int64_t ld_k, int64_t ld_v, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(n, THREADS * PASSES, attr, s);
    return cudaLaunchKernelEx(&cfg, paged_append_kernel<DT, Q8, PASSES>, k, v, ld_k, ld_v, n, row_start,
                              paged_view(c, pg), pool_of(c, layer, 8));
}
template <int DT, bool Q8>
cudaError_t append_t(const kvc_cache &c, const kvc_pages &pg, int layer, const int32_t *row_start, int n_rows,
                     const void *k, const void *v, int64_t ld_k, int64_t ld_v, cudaStream_t s) {
    const int per_row = c.d.n_head_kv * (c.d.head_dim / 8);
    const int64_t n = (int64_t)n_rows * per_row;
    return many(n, APPEND_PASSES)
               ? append_p<DT, Q8, APPEND_PASSES>(c, pg, layer, row_start, n, k, v, ld_k, ld_v, s)
               : append_p<DT, Q8, 1>(c, pg, layer, row_start, n, k, v, ld_k, ld_v, s);
}

template <int DT, bool Q8, int PASSES, bool WIDE>
cudaError_t read_p(const kvc_cache &c, const kvc_pages &pg, int layer, const int32_t *row_start, int64_t n,
                   void *k, void *v, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(n, THREADS * PASSES, attr, s);
    return cudaLaunchKernelEx(&cfg, paged_read_kernel<DT, Q8, PASSES, WIDE>, k, v, n, row_start,
                              paged_view(c, pg), pool_of(c, layer, Q8 ? 16 : 8));
}
template <int DT, bool Q8>
cudaError_t read_t(const kvc_cache &c, const kvc_pages &pg, int layer, const int32_t *row_start, int n_rows, void *k,
                   void *v, cudaStream_t s) {
    const int per_row = c.d.n_head_kv * (c.d.head_dim / (Q8 ? 16 : 8));
    const int64_t n = (int64_t)n_rows * per_row;
    const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0;
    // 16-byte stores elsewhere: 69 us instead of 57 for the q8_0 read above
    if (!wide) return read_p<DT, Q8, 1, false>(c, pg, layer, row_start, n, k, v, s);
    return many(n, READ_PASSES<Q8>) ? read_p<DT, Q8, READ_PASSES<Q8>, true>(c, pg, layer, row_start, n, k, v, s)
                                    : read_p<DT, Q8, 1, true>(c, pg, layer, row_start, n, k, v, s);
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
