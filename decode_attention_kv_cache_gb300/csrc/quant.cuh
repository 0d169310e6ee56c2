// The q8_0 block quantiser and the input loader, shared by the append kernel and the fused decode and
// prefill steps so that all of them store the same bytes.
//
// One block is 32 values along head_dim: fp16 scale d = amax / 127, int8 codes q = round(x / d)
// (llama.cpp PR #58 "completion : allow the prompt to be processed under its own split mode",
// section "Why": the q8_0 device-resident cache).  The arithmetic repeats, bit for bit, the float32
// op order: amax exact, d = amax/127 and x/d by IEEE division, ties away from zero.  The quotient x/d
// is taken as x times the IEEE reciprocal of d and rounded with a 1.5*2^23 shift; that product is
// within 5e-5 of the IEEE quotient, so the rounded code can differ from round(x/d) only when the
// product lies within that distance of a .5 boundary, and exactly those values are recomputed with
// the IEEE division (both values of a pair, the one away from the boundary giving the same code
// either way).  A non-finite block (outside the method's domain) gets zero codes.
#pragma once

#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "ptx.cuh"

namespace kvc {

// 8 consecutive input values (f32, bf16 or f16: DT is a kvc_dtype) as they lie in memory.
template <int DT>
struct Raw8 {
    uint4 u[DT == KVC_IN_F32 ? 2 : 1];
};

// Those from element index idx, read through L2 (a kernel just before the reader may have written them).
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const void *base, int64_t idx) {
    Raw8<DT> r;
    if constexpr (DT == KVC_IN_F32) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + idx);
        r.u[0] = __ldcg(p);
        r.u[1] = __ldcg(p + 1);
    } else {
        r.u[0] = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + idx));
    }
    return r;
}

// As floats: bf16 and f16 widen exactly.
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT> &r, float (&x)[8]) {
    if constexpr (DT == KVC_IN_F32) {
        const uint4 a = r.u[0], b = r.u[1];
        x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
        x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y); x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
    } else {
        const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == KVC_IN_BF16) {
                x[2 * i] = __uint_as_float(w[i] << 16);          // the bf16 bits are the f32's top half
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                x[2 * i] = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xFFFF)));
                x[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ void load_inputs8(const void *base, int64_t idx, float (&x)[8]) {
    widen8<DT>(load_raw8<DT>(base, idx), x);
}

// The codes of a block whose d is 2^-128 or less, so that 1 / d would be infinite, and so coarse that x / d may pass 127.
// Not inlined: its divisions would cost the ordinary blocks' code registers.
static __device__ __noinline__ void q8_0_coarse32(const float *x, float d, uint32_t *packed) {
#pragma unroll 1
    for (int w = 0; w < 8; ++w) {
        packed[w] = 0u;
#pragma unroll 1
        for (int b = 0; b < 4; ++b)
            packed[w] |= ((uint32_t)max(min((int)roundf(__fdiv_rn(x[4 * w + b], d)), 127), -127) & 0xFFu) << (8 * b);
    }
}

// Quantise x[0..31]: the 32 codes packed four to a word (byte i of word w is code 4 w + i) and the
// fp16 bits of the scale.
__device__ __forceinline__ uint16_t q8_0_quantize32(const float (&x)[32], uint32_t (&packed)[8]) {
    float m2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        m2[0] = ptx::fmax3(m2[0], fabsf(x[i]), fabsf(x[i + 1]));
        m2[1] = ptx::fmax3(m2[1], fabsf(x[i + 2]), fabsf(x[i + 3]));
    }
    const float amax = fmaxf(m2[0], m2[1]);
    const float d = __fdiv_rn(amax, 127.0f);
#pragma unroll
    for (int w = 0; w < 8; ++w) packed[w] = 0u;
    // codes are zero when amax/127 is zero (x/d undefined); |x * r| <= 127 (to an ulp) otherwise
    if (__builtin_expect(d > 0.f && d <= 0x1p-128f, 0)) {
        float z[32];
        uint32_t w8[8];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = x[i];
        q8_0_coarse32(z, d, w8);
#pragma unroll
        for (int w = 0; w < 8; ++w) packed[w] = w8[w];
    } else if (d > 0.f && amax <= 3.402823466e38f) {
        const float r = __frcp_rn(d);
        const uint64_t r2 = ptx::f2_pack(r, r), mz = ptx::f2_pack(-0.f, -0.f), M2 = ptx::f2_pack(12582912.f, 12582912.f),
                       nM2 = ptx::f2_pack(-12582912.f, -12582912.f), n1 = ptx::f2_pack(-1.f, -1.f);
        int q[32];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const uint64_t y = ptx::f2_fma(ptx::f2_pack(x[i], x[i + 1]), r2, mz);   // x * r, one rounding
            const uint64_t t = ptx::f2_add(y, M2);                                // y rounded to an integer (to even)
            const uint64_t f = ptx::f2_fma(ptx::f2_add(t, nM2), n1, y);              // y minus that integer
            float t0, t1, f0, f1;
            ptx::f2_unpack(t, t0, t1);
            ptx::f2_unpack(f, f0, f1);
            q[i] = __float_as_int(t0) - 0x4B400000;
            q[i + 1] = __float_as_int(t1) - 0x4B400000;
            if (fmaxf(fabsf(f0), fabsf(f1)) > 0.4999f) {  // near a tie: exact quotients
                q[i] = (int)roundf(__fdiv_rn(x[i], d));
                q[i + 1] = (int)roundf(__fdiv_rn(x[i + 1], d));
            }
        }
#pragma unroll
        for (int w = 0; w < 8; ++w)
            packed[w] = __byte_perm(__byte_perm(q[4 * w], q[4 * w + 1], 0x0040),
                                    __byte_perm(q[4 * w + 2], q[4 * w + 3], 0x0040), 0x5410);
    }
    return __half_as_ushort(__float2half_rn(d));
}

// The code of |x| / d for a pair of values, exact, without a division: round(fl(|x| / d)), ties away from zero.
// k is an integer with k <= |x| / d < k + 1 but for an error that does not matter (at an integer either choice of
// k leads to the same code), h = k + 1/2.  The rounded quotient reaches h exactly where |x| / d is not below the
// middle between h and the float before it, h - 2^(j - 24) with 2^j <= h < 2^(j + 1): a tie there goes to h, whose
// last mantissa bits are zero.  Near h the residue |x| - h d is exact (both are multiples of half a unit in the
// last place of d, and so is their difference of a few thousand of those), so the sign of
// |x| - h d + 2^(j - 24) d, one more rounding, decides.  (At h = 1/2 the floats below h are half as far apart; no
// residue lies between the two limits.)  d24 = d 2^-24 has to be a normal number.  The codes are the low bytes.
__device__ __forceinline__ void q8_0_exact2(float x0, float x1, uint64_t r2, uint64_t d2, uint64_t d24_2, uint32_t &q0,
                                            uint32_t &q1) {
    const uint64_t a = ptx::f2_pack(fabsf(x0), fabsf(x1)), M2 = ptx::f2_pack(12582912.f, 12582912.f),
                   nM2 = ptx::f2_pack(-12582912.f, -12582912.f), n1 = ptx::f2_pack(-1.f, -1.f),
                   nh = ptx::f2_pack(-0.5f, -0.5f);
    const uint64_t t = ptx::f2_add(ptx::f2_fma(a, r2, nh), M2);                 // k + M
    const uint64_t h = ptx::f2_fma(ptx::f2_add(t, nM2), n1, nh);                // -(k + 1/2)
    float h0, h1, c0, c1, t0, t1;
    ptx::f2_unpack(h, h0, h1);
    const uint64_t j = ptx::f2_pack(__uint_as_float(__float_as_uint(h0) & 0x7F800000u),
                                    __uint_as_float(__float_as_uint(h1) & 0x7F800000u));
    ptx::f2_unpack(ptx::f2_fma(j, d24_2, ptx::f2_fma(h, d2, a)), c0, c1);
    ptx::f2_unpack(t, t0, t1);
    const int s0 = __float_as_int(x0) >> 31, s1 = __float_as_int(x1) >> 31;
    q0 = (uint32_t)(((__float_as_int(t0) + 1 + (__float_as_int(c0) >> 31)) ^ s0) - s0);
    q1 = (uint32_t)(((__float_as_int(t1) + 1 + (__float_as_int(c1) >> 31)) ^ s1) - s1);
}

// A block spread over four neighbouring lanes, eight values each: this lane's codes and the block's scale.  All four
// lanes take part.  The same codes as above; with eight values to a thread one look at all of them for a near tie is
// cheaper than one for each pair, and bf16 and fp16 inputs, whose quotients have few bits, meet ties in half of the
// warps, so the exact codes come from q8_0_exact2 and not from divisions.  rcp.approx is within one unit
// in the last place, so x * r is within 127 * (2^-23 + 2^-24) = 2.3e-5 of x / d.
__device__ __forceinline__ uint16_t q8_0_quantize_quad(const float (&x)[8], uint32_t (&packed)[2]) {
    float m = ptx::fmax3(fabsf(x[0]), fabsf(x[1]), fabsf(x[2]));
    m = ptx::fmax3(m, fabsf(x[3]), fabsf(x[4]));
    m = ptx::fmax3(m, fabsf(x[5]), fabsf(x[6]));
    m = fmaxf(m, fabsf(x[7]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float d = __fdiv_rn(m, 127.0f);
    packed[0] = packed[1] = 0u;
    if (d > 0.f && m <= 3.402823466e38f) {
        uint32_t q[8];   // the code is the low byte
        if (d >= 1e-30f) {
            float r;
            asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
            const uint64_t r2 = ptx::f2_pack(r, r), mz = ptx::f2_pack(-0.f, -0.f),
                           M2 = ptx::f2_pack(12582912.f, 12582912.f), nM2 = ptx::f2_pack(-12582912.f, -12582912.f),
                           n1 = ptx::f2_pack(-1.f, -1.f);
            float off = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const uint64_t y = ptx::f2_fma(ptx::f2_pack(x[i], x[i + 1]), r2, mz);   // x * r, one rounding
                const uint64_t t = ptx::f2_add(y, M2);                            // y rounded to an integer (to even)
                const uint64_t f = ptx::f2_fma(ptx::f2_add(t, nM2), n1, y);          // y minus that integer
                float t0, t1, f0, f1;
                ptx::f2_unpack(t, t0, t1);
                ptx::f2_unpack(f, f0, f1);
                q[i] = __float_as_uint(t0);   // 1.5 * 2^23 plus the code
                q[i + 1] = __float_as_uint(t1);
                off = ptx::fmax3(off, fabsf(f0), fabsf(f1));
            }
            if (off > 0.4999f) {  // near a tie
                const uint64_t d2 = ptx::f2_pack(d, d), d24_2 = ptx::f2_pack(d * 0x1p-24f, d * 0x1p-24f);
#pragma unroll
                for (int i = 0; i < 8; i += 2) q8_0_exact2(x[i], x[i + 1], r2, d2, d24_2, q[i], q[i + 1]);
            }
        } else {   // 1 / d or d 2^-24 may leave the normal range, and a subnormal d be so coarse that x / d passes 127
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                float v = x[0];
#pragma unroll
                for (int j = 1; j < 8; ++j) v = i == j ? x[j] : v;
                const uint32_t c = (uint32_t)max(min((int)roundf(__fdiv_rn(v, d)), 127), -127);
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = i == j ? c : q[j];
            }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w)
            packed[w] = __byte_perm(__byte_perm(q[4 * w], q[4 * w + 1], 0x0040),
                                    __byte_perm(q[4 * w + 2], q[4 * w + 3], 0x0040), 0x5410);
    }
    return __half_as_ushort(__float2half_rn(d));
}

}  // namespace kvc
