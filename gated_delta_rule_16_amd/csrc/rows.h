// Rows of channels in fp32 or bf16, read and written E channels at a time by
// kernels that take the type at run time (one uniform branch per access).
//
// A full group of E channels is one vector access (16 bytes for 8 bf16 or 4
// fp32).  The types below carry element alignment only: gfx950 executes
// global vector accesses at any element-aligned address, so rows of odd
// length, slices of a wider projection and unaligned bases take the same
// instructions as aligned ones.  The last, partial group of a row goes
// element by element.
#pragma once

#include "gdr_device.h"
#include "mfma_common.h"

namespace gdr {

typedef uint32_t u32x2_e2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_e2 __attribute__((aligned(2)));
typedef uint32_t u32x2_e4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));

// E channels as loaded: fp32 uses all E words, bf16 the first half.
template <int E> struct RawRow { uint32_t w[E]; };

// Loads channels [0, valid) of the E at element offset `off` (64-bit) from
// `base`; the others become 0.  valid may be negative.
template <int E>
__device__ __forceinline__ void row_load(RawRow<E>& r, const void* base, int64_t off, bool bf16,
                                         int valid) {
    if (valid >= E) {
        if (bf16) {
            const bf16_t* p = static_cast<const bf16_t*>(base) + off;
            if constexpr (E == 8) {
                const u32x4_e2 v = *reinterpret_cast<const u32x4_e2*>(p);
                r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
            } else if constexpr (E == 4) {
                const u32x2_e2 v = *reinterpret_cast<const u32x2_e2*>(p);
                r.w[0] = v.x; r.w[1] = v.y;
            } else if constexpr (E == 2) {
                r.w[0] = *reinterpret_cast<const u32_e2*>(p);
            } else {
                static_assert(E == 1, "group size");
                r.w[0] = *p;
            }
        } else {
            const float* p = static_cast<const float*>(base) + off;
            if constexpr (E >= 4) {
#pragma unroll
                for (int i = 0; i < E; i += 4) {
                    const u32x4_e4 v = *reinterpret_cast<const u32x4_e4*>(p + i);
                    r.w[i] = v.x; r.w[i + 1] = v.y; r.w[i + 2] = v.z; r.w[i + 3] = v.w;
                }
            } else if constexpr (E == 2) {
                const u32x2_e4 v = *reinterpret_cast<const u32x2_e4*>(p);
                r.w[0] = v.x; r.w[1] = v.y;
            } else {
                r.w[0] = __float_as_uint(*p);
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) r.w[e] = 0u;
    if (bf16) {
        const bf16_t* p = static_cast<const bf16_t*>(base) + off;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < valid) r.w[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
    } else {
        const float* p = static_cast<const float*>(base) + off;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < valid) r.w[e] = __float_as_uint(p[e]);
    }
}

template <int E>
__device__ __forceinline__ void row_unpack(float (&f)[E], const RawRow<E>& r, bool bf16) {
    if (bf16) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            f[e] = __uint_as_float((e & 1) ? (r.w[e / 2] & 0xffff0000u) : (r.w[e / 2] << 16));
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = __uint_as_float(r.w[e]);
    }
}

// Stores channels [0, valid) of the E (bf16: round to nearest even).
template <int E>
__device__ __forceinline__ void row_store(void* base, int64_t off, bool bf16, const float (&f)[E],
                                          int valid) {
    if (bf16) {
        bf16_t* p = static_cast<bf16_t*>(base) + off;
        if (valid >= E) {
            if constexpr (E == 8) {
                *reinterpret_cast<u32x4_e2*>(p) = u32x4_e2{cvt_pk(f[0], f[1]), cvt_pk(f[2], f[3]),
                                                           cvt_pk(f[4], f[5]), cvt_pk(f[6], f[7])};
            } else if constexpr (E == 4) {
                *reinterpret_cast<u32x2_e2*>(p) = u32x2_e2{cvt_pk(f[0], f[1]), cvt_pk(f[2], f[3])};
            } else if constexpr (E == 2) {
                *reinterpret_cast<u32_e2*>(p) = cvt_pk(f[0], f[1]);
            } else {
                *p = f2bf(f[0]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < valid) p[e] = f2bf(f[e]);
        }
    } else {
        float* p = static_cast<float*>(base) + off;
        if (E >= 4 && valid >= E) {
#pragma unroll
            for (int i = 0; i + 3 < E; i += 4)
                *reinterpret_cast<f32x4_e4*>(p + i) = f32x4_e4{f[i], f[i + 1], f[i + 2], f[i + 3]};
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < valid) p[e] = f[e];
        }
    }
}

// M consecutive floats (M a multiple of 4) of a parameter; beyond `valid`: 0.
template <int M>
__device__ __forceinline__ void param_load(float (&f)[M], const float* p, int valid) {
    static_assert(M % 4 == 0, "groups of 4");
    if (valid >= M) {
#pragma unroll
        for (int i = 0; i < M; i += 4) {
            const f32x4_e4 v = *reinterpret_cast<const f32x4_e4*>(p + i);
            f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i) f[i] = i < valid ? p[i] : 0.f;
    }
}

constexpr float kLog2e = 1.44269504088896f;
constexpr float kLn2 = 0.693147180559945f;

// exp(x) for x <= 0, relative error ~2^-23 also at large |x|: the rounding
// of x log2(e) (up to |x| 2^-24, which exp would turn into a relative error
// |x| 2^-24) is recovered with an fma and applied to first order.
__device__ __forceinline__ float exp_neg(float x) {
    const float p = x * kLog2e;
    float r = __builtin_fmaf(x, kLog2e, -p);
    r = __builtin_fmaf(x, 1.925963033500117e-8f, r);      // log2(e) - fl(log2(e))
    const float e = __builtin_amdgcn_exp2f(p);
    // p below the exponent range: e is 0, and r may be inf - inf
    return p > -149.f ? __builtin_fmaf(e, r * kLn2, e) : (p != p ? p : 0.f);
}

// log(1 + e) for e in [0, 1]: 2 atanh(s) with s = e / (2 + e) <= 1/3, the
// odd series to s^17 (its remainder is below 2^-27 of the sum at s = 1/3).
// Relative error stays ~2^-23 for small e, where log(1 + e) would lose it.
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = e * __builtin_amdgcn_rcpf(2.f + e);
    const float q = s * s;
    float c = 1.f / 17.f;
    c = __builtin_fmaf(c, q, 1.f / 15.f);
    c = __builtin_fmaf(c, q, 1.f / 13.f);
    c = __builtin_fmaf(c, q, 1.f / 11.f);
    c = __builtin_fmaf(c, q, 1.f / 9.f);
    c = __builtin_fmaf(c, q, 1.f / 7.f);
    c = __builtin_fmaf(c, q, 1.f / 5.f);
    c = __builtin_fmaf(c, q, 1.f / 3.f);
    c = c * q;
    return 2.f * __builtin_fmaf(s, c, s);
}

// 1 / (1 + exp(-x)); 0 and 1 at the ends of the range, NaN for NaN.
__device__ __forceinline__ float sigmoid(float x) {
    const float e = exp_neg(-fabsf(x));
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    return x >= 0.f ? r : e * r;
}

// softplus(x) = max(x, 0) + log(1 + exp(-|x|)), and its derivative.
__device__ __forceinline__ float softplus(float x) {
    const float l = log1p_unit(exp_neg(-fabsf(x)));
    return x > 0.f ? x + l : l;
}

}  // namespace gdr
