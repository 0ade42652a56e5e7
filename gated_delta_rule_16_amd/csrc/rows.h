// Rows of channels in fp32 or bf16, read and written E channels at a time.
//
// A full group of E channels is one vector access (16 bytes for 8 bf16 or 4
// fp32).  The types below carry element alignment only: gfx950 executes
// global vector accesses at any element-aligned address, so slices of a wider
// projection and unaligned bases take the same instructions as aligned ones.
//
// A load that is in flight must not meet a branch that merges its register
// with another value: the merge is a copy, and the copy waits for the load.
// So the type is a template parameter, a group's words are written by its
// load alone (lanes without a group keep the zeros set before it), and in the
// RAG variant the elements of a partial group have registers of their own,
// joined at unpacking.  The variant is for the shortest rows: elsewhere the
// last group of a row of any length is moved back to end with the row, and
// the channels that it then shares with the group before it are worked on
// twice, to the same result.
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

template <int E, bool BF16, bool RAG> struct Row {
    static constexpr int W = BF16 ? (E + 1) / 2 : E;
    uint32_t w[W];              // the vector access
    uint32_t p[RAG ? E : 1];    // a partial group's elements

    // Channels [0, valid) at element offset `off`; the others become 0.  Without
    // RAG valid is 0 or E.
    __device__ __forceinline__ void load(const void* base, int64_t off, int valid) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0u;
        if (valid >= E) {
            if constexpr (BF16) {
                const bf16_t* q = static_cast<const bf16_t*>(base) + off;
                if constexpr (E == 8) {
                    const u32x4_e2 v = *reinterpret_cast<const u32x4_e2*>(q);
                    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
                } else if constexpr (E == 4) {
                    const u32x2_e2 v = *reinterpret_cast<const u32x2_e2*>(q);
                    w[0] = v.x; w[1] = v.y;
                } else if constexpr (E == 2) {
                    w[0] = *reinterpret_cast<const u32_e2*>(q);
                } else {
                    static_assert(E == 1, "group size");
                    w[0] = *q;
                }
            } else {
                const float* q = static_cast<const float*>(base) + off;
                if constexpr (E >= 4) {
#pragma unroll
                    for (int i = 0; i < E; i += 4) {
                        const u32x4_e4 v = *reinterpret_cast<const u32x4_e4*>(q + i);
                        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
                    }
                } else if constexpr (E == 2) {
                    const u32x2_e4 v = *reinterpret_cast<const u32x2_e4*>(q);
                    w[0] = v.x; w[1] = v.y;
                } else {
                    w[0] = __float_as_uint(*q);
                }
            }
        }
        if constexpr (RAG) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                p[e] = 0u;
                if (valid < E && e < valid) {
                    if constexpr (BF16)
                        p[e] = static_cast<const bf16_t*>(base)[off + e];
                    else
                        p[e] = __float_as_uint(static_cast<const float*>(base)[off + e]);
                }
            }
        }
    }

    // The same channels to memory, bit for bit (a store of the unpacked values
    // would make signalling NaNs quiet).
    __device__ __forceinline__ void copy_to(void* base, int64_t off, int valid) const {
        static_assert(E == 4 || E == 8, "group size");
        if (valid >= E) {
            if constexpr (BF16) {
                bf16_t* q = static_cast<bf16_t*>(base) + off;
                if constexpr (E == 8)
                    *reinterpret_cast<u32x4_e2*>(q) = u32x4_e2{w[0], w[1], w[2], w[3]};
                else
                    *reinterpret_cast<u32x2_e2*>(q) = u32x2_e2{w[0], w[1]};
            } else {
                uint32_t* q = static_cast<uint32_t*>(base) + off;
#pragma unroll
                for (int i = 0; i < E; i += 4)
                    *reinterpret_cast<u32x4_e4*>(q + i) =
                        u32x4_e4{w[i], w[i + 1], w[i + 2], w[i + 3]};
            }
        }
        if constexpr (RAG) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (valid < E && e < valid) {
                    if constexpr (BF16)
                        static_cast<bf16_t*>(base)[off + e] = (bf16_t)p[e];
                    else
                        static_cast<uint32_t*>(base)[off + e] = p[e];
                }
            }
        }
    }

    __device__ __forceinline__ void unpack(float (&f)[E]) const {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (BF16)
                f[e] = __uint_as_float((e & 1) ? (w[e / 2] & 0xffff0000u) : (w[e / 2] << 16));
            else
                f[e] = __uint_as_float(w[e]);
        }
        if constexpr (RAG) {
            // one of the two is 0
#pragma unroll
            for (int e = 0; e < E; ++e)
                f[e] = __uint_as_float(__float_as_uint(f[e]) | (BF16 ? p[e] << 16 : p[e]));
        }
    }
};

// Stores channels [0, valid) of the E (bf16: round to nearest even).  Without
// RAG valid is 0 or E.
template <int E, bool RAG = true>
__device__ __forceinline__ void row_store(void* base, int64_t off, bool bf16, const float (&f)[E],
                                          int valid) {
    if (valid >= E) {
        if (bf16) {
            bf16_t* p = static_cast<bf16_t*>(base) + off;
            if constexpr (E == 8)
                *reinterpret_cast<u32x4_e2*>(p) = u32x4_e2{cvt_pk(f[0], f[1]), cvt_pk(f[2], f[3]),
                                                           cvt_pk(f[4], f[5]), cvt_pk(f[6], f[7])};
            else if constexpr (E == 4)
                *reinterpret_cast<u32x2_e2*>(p) = u32x2_e2{cvt_pk(f[0], f[1]), cvt_pk(f[2], f[3])};
            else if constexpr (E == 2)
                *reinterpret_cast<u32_e2*>(p) = cvt_pk(f[0], f[1]);
            else
                *p = f2bf(f[0]);
        } else {
            float* p = static_cast<float*>(base) + off;
            if constexpr (E >= 4) {
#pragma unroll
                for (int i = 0; i < E; i += 4)
                    *reinterpret_cast<f32x4_e4*>(p + i) =
                        f32x4_e4{f[i], f[i + 1], f[i + 2], f[i + 3]};
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) p[e] = f[e];
            }
        }
        return;
    }
    if constexpr (RAG) {
        if (bf16) {
            bf16_t* p = static_cast<bf16_t*>(base) + off;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < valid) p[e] = f2bf(f[e]);
        } else {
            float* p = static_cast<float*>(base) + off;
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

// The same for any M.
template <int M>
__device__ __forceinline__ void small_load(float (&f)[M], const float* p, int valid) {
    if constexpr (M % 4 == 0) {
        param_load<M>(f, p, valid);
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i) f[i] = i < valid ? p[i] : 0.f;
    }
}

constexpr float kLog2e = 1.44269504088896f;
constexpr float kLn2 = 0.693147180559945f;

// exp(-|x|), 0 far down.  The argument's rounding makes its relative error
// |x| 2^-24 (2^-21 at x = -8): no more than the sum dt + dt_bias in front of a
// softplus has rounded off already.
__device__ __forceinline__ float exp_neg_abs(float x) {
    return __builtin_amdgcn_exp2f(fabsf(x) * -kLog2e);
}

// log(1 + e) for e in [0, 1] as e times a polynomial of degree 9 (fitted for
// the smallest relative error over [0, 1]: 1.2e-8 with these coefficients, 1.3e-7
// as evaluated).  Relative error stays ~2^-23 for small e, where log(1 + e)
// would lose it, and no transcendental is used.
__device__ __forceinline__ float log1p_unit(float e) {
    float c = -0.00324386684f;
    c = __builtin_fmaf(c, e, 0.0198507495f);
    c = __builtin_fmaf(c, e, -0.0569581948f);
    c = __builtin_fmaf(c, e, 0.106035195f);
    c = __builtin_fmaf(c, e, -0.153055131f);
    c = __builtin_fmaf(c, e, 0.19675912f);
    c = __builtin_fmaf(c, e, -0.249541283f);
    c = __builtin_fmaf(c, e, 0.333299607f);
    c = __builtin_fmaf(c, e, -0.499999017f);
    c = __builtin_fmaf(c, e, 1.f);
    return c * e;
}

// 1 / (1 + exp(-x)), relative error (1 - sigmoid) |x| 2^-24 and a few steps.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -kLog2e));
}

// softplus(x) = max(x, 0) + log(1 + exp(-|x|)); NaN stays NaN.
__device__ __forceinline__ float softplus(float x) {
    return (x < 0.f ? 0.f : x) + log1p_unit(exp_neg_abs(x));
}

// softplus(x) and its derivative sigmoid(x), from one exp.
__device__ __forceinline__ void softplus_grad(float x, float& y, float& dy) {
    const float e = exp_neg_abs(x);
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    y = (x < 0.f ? 0.f : x) + log1p_unit(e);
    dy = x < 0.f ? e * r : r;
}

}  // namespace gdr
