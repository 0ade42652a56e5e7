// The chain of linear attention (see linear_attn.hip): operand fragments, tiles in
// LDS and the chunk kernel.
#pragma once

#include "linear_launch.h"
#include "mfma_common.h"
#include "rows.h"

namespace gdr {
namespace la {

constexpr int ZB = 64;              // channels of z and out per workgroup
constexpr float kLeast = -1e4f;     // log decays from here on are a reset: exp is 0

// 16-byte pieces of a tile's row are permuted by the row, so that rows read at one
// column, and 4x4 blocks read transposed, meet different banks.
__device__ __forceinline__ int swz(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }

// bf16 inputs: chunks of 64 tokens on the bf16 matrix cores.  A computed operand
// enters as NT bf16 terms (24 bits with three).
struct Bf16 {
    typedef bf16_t T;
    static constexpr bool is_bf16 = true;
    static constexpr int C = 64;
    static constexpr int EP = 8;    // elements per 16 bytes
    static constexpr int NT = 3;
    typedef bf16x8 Frag;
    struct Terms {
        bf16x8 t[NT];
    };
    static __device__ __forceinline__ void split(const f32x8& x, Terms& o) {
        uint32_t w[NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                w[n][i] = cvt_pk(a, b);
                if (n + 1 < NT) {
                    a -= __uint_as_float(w[n][i] << 16);
                    b -= __uint_as_float(w[n][i] & 0xffff0000u);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
            o.t[n] = __builtin_bit_cast(bf16x8, u32x4{w[n][0], w[n][1], w[n][2], w[n][3]});
    }
    static __device__ __forceinline__ f32x8 widen(const Frag& f) {
        const u32x4 w = __builtin_bit_cast(u32x4, f);
        f32x8 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[2 * i] = __uint_as_float(w[i] << 16);
            r[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        return r;
    }
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, const f32x4& c) {
        return mfma16(a, b, c);
    }
    // the smallest terms first
    static __device__ __forceinline__ f32x4 mma(const Terms& a, const Frag& b, f32x4 c) {
#pragma unroll
        for (int n = NT - 1; n >= 0; --n) c = mfma16(a.t[n], b, c);
        return c;
    }
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Terms& b, f32x4 c) {
#pragma unroll
        for (int n = NT - 1; n >= 0; --n) c = mfma16(a, b.t[n], c);
        return c;
    }
};

// fp32 inputs: chunks of 32 tokens on the fp32 matrix cores.  A lane's 8 elements of
// a 32-deep contraction go in one at a time: the contraction's order is free.
struct F32 {
    typedef float T;
    static constexpr bool is_bf16 = false;
    static constexpr int C = 32;
    static constexpr int EP = 4;
    static constexpr int NT = 1;
    typedef f32x8 Frag;
    struct Terms {
        f32x8 t[1];
    };
    static __device__ __forceinline__ void split(const f32x8& x, Terms& o) { o.t[0] = x; }
    static __device__ __forceinline__ f32x8 widen(const Frag& f) { return f; }
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = mfma_f32(a[i], b[i], c);
        return c;
    }
    static __device__ __forceinline__ f32x4 mma(const Terms& a, const Frag& b, const f32x4& c) {
        return mma(a.t[0], b, c);
    }
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Terms& b, const f32x4& c) {
        return mma(a, b.t[0], c);
    }
};

// A tile of rows of W elements in LDS.
template <class P, int W> struct Tile {
    typedef typename P::T T;
    static constexpr int PPR = W / P::EP;           // 16-byte pieces per row
    static __device__ __forceinline__ T* piece(T* t, int row, int c) {
        return t + row * W + ((c ^ (swz(row) & (PPR - 1))) * P::EP);
    }
    static __device__ __forceinline__ const T* piece(const T* t, int row, int c) {
        return t + row * W + ((c ^ (swz(row) & (PPR - 1))) * P::EP);
    }
    // elements 8 c8 .. 8 c8 + 7 of a row
    static __device__ __forceinline__ typename P::Frag row8(const T* t, int row, int c8) {
        if constexpr (P::is_bf16) {
            return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(piece(t, row, c8)));
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4*>(piece(t, row, 2 * c8));
            const f32x4 b = *reinterpret_cast<const f32x4*>(piece(t, row, 2 * c8 + 1));
            return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        }
    }
    // rows row0 + 8 g .. + 7 of one column per lane m, which is
    // col0 + step (m / 4) + m % 4 (g = lane / 16, m = lane % 16)
    static __device__ __forceinline__ typename P::Frag col8(const T* t, int lane, int row0,
                                                            int col0, int step) {
        const int g = lane >> 4, m = lane & 15;
        if constexpr (P::is_bf16) {
            // lane 4 r + c of a group points at 4 columns of row r (lds_tr16)
            const int r = row0 + 8 * g + (m >> 2), c = col0 + step * (m & 3);
            const s16x4 a = lds_tr16(piece(t, r, c >> 3) + (c & 7));
            const s16x4 b = lds_tr16(piece(t, r + 4, c >> 3) + (c & 7));
            typedef short s16x8 __attribute__((ext_vector_type(8)));
            const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            return __builtin_bit_cast(bf16x8, v);
        } else {
            const int c = col0 + step * (m >> 2) + (m & 3);
            f32x8 v;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = row0 + 8 * g + i;
                v[i] = *(piece(t, r, c >> 2) + (c & 3));
            }
            return v;
        }
    }
};

// The pieces of a [C, W] tile that one of 256 threads moves from memory.
template <class P, int W> struct Stage {
    static constexpr int PPR = W / P::EP;
    static constexpr int N = P::C * PPR / 256;
    u32x4 w[N];
    // Rows are tokens t, t + dir, ..; rows from len on and channels from `width` on
    // become 0.  `base`: of token 0.
    __device__ __forceinline__ void load(const void* base, int64_t t, int dir, int64_t st, int len,
                                         int width, int tid) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = tid + 256 * i, row = id / PPR, c = id % PPR;
            w[i] = u32x4{0u, 0u, 0u, 0u};
            if (row < len && c * P::EP < width) {
                const typename P::T* p = static_cast<const typename P::T*>(base) +
                                         (t + dir * row) * st + c * P::EP;
                if constexpr (P::is_bf16)
                    w[i] = *reinterpret_cast<const u32x4_e2*>(p);
                else
                    w[i] = *reinterpret_cast<const u32x4_e4*>(p);
            }
        }
    }
    __device__ __forceinline__ void put(typename P::T* tile, int tid) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = tid + 256 * i, row = id / PPR, c = id % PPR;
            *reinterpret_cast<u32x4*>(Tile<P, W>::piece(tile, row, c)) = w[i];
        }
    }
    // Whether an element is infinite or no number.
    __device__ __forceinline__ bool bad() const {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t v = w[i][j];
                if constexpr (P::is_bf16) {
                    any |= (v & 0x7f80u) == 0x7f80u;
                    any |= (v & 0x7f800000u) == 0x7f800000u;
                } else {
                    any |= (v & 0x7f800000u) == 0x7f800000u;
                }
            }
        return any != 0;
    }
};

// Where a workgroup works: the (sequence, head, segment) groups go round the 8 XCDs,
// and all jobs and channel blocks of one group stay on one, whose L2 they share.
struct Place {
    int64_t b, h, seg;
    int job, zb;
};

__device__ __forceinline__ bool place(const LaChain& a, int64_t id, Place& o) {
    int nz[3], per = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        nz[j] = j < a.njobs ? (a.job[j].zd + ZB - 1) / ZB : 0;
        per += nz[j];
    }
    const int64_t grp = id / (8 * per) * 8 + id % 8;
    int k = (int)(id / 8 % per);
    if (grp >= a.B * a.H * a.nseg) return false;
    o.job = 0;
    while (k >= nz[o.job]) k -= nz[o.job++];
    o.zb = k;
    o.h = grp % a.H;
    o.b = grp / a.H % a.B;
    o.seg = grp / a.H / a.B;
    return true;
}

__device__ __forceinline__ const void* head_base(const LaTensor& t, int64_t b, int64_t h,
                                                 size_t elem) {
    return static_cast<const char*>(t.p) + (b * t.sb + h / t.share * t.sh) * elem;
}

// Log decay (base 2) that the state goes through before token t is added.
__device__ __forceinline__ double decay2(const LaChain& a, int64_t b, int64_t h, int64_t t) {
    if (!a.g || t >= a.T) return 0.0;
    float g = a.g_head ? a.g[h] : a.g[(b * a.T + t) * a.H + h];
    g = g < kLeast ? kLeast : g;
    return (double)g * 1.4426950408889634;
}

}  // namespace la
}  // namespace gdr
