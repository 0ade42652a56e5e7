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

// Tiles in LDS.  The 16-byte pieces of a row are permuted by the row so that operands
// meet different banks (64 of 4 bytes).  Rows read 16 bytes a lane go by lanes 0-3,
// 12-15, 20-23 and 24-27, then 4-11, 16-19 and 28-31, and so on; blocks read
// transposed, 8 bytes a lane, go by lanes 0-31 and 32-63.  With one order of 8 rows for
// all kinds 868 of 2474 LDS cycles a chunk were conflicts; with these, none in the
// kernel of the states alone and 500 of 2940 in the chain's, whose time LDS does not
// decide.
enum TileKind {
    ROWS,       // read by rows only
    BOTH        // by rows, and transposed, 16 neighbouring columns at once
};

// A computed operand of a product: N bf16 terms, the largest first (or fp32 itself).
template <class F, int N> struct Terms {
    F t[N];
};

// bf16 inputs: chunks of 64 tokens on the bf16 matrix cores.  A computed operand of the
// state enters as three bf16 terms (24 bits); one of out as NO terms: three, or two
// (2^-17 of the operand) where out is rounded to bf16, 2^-9 of itself.
template <int NO_> struct Bf16 {
    typedef bf16_t T;
    static constexpr bool is_bf16 = true;
    static constexpr int C = 64;
    static constexpr int EP = 8;    // elements per 16 bytes
    static constexpr int NO = NO_, NS = 3;
    typedef bf16x8 Frag;
    // x in N terms each.  The residuals x - hi come from dot products of the packed
    // terms with (-1, 0) and (0, -1), exact as in split2.
    template <int N>
    static __device__ __forceinline__ void split_pair(float a, float b, uint32_t (&w)[N]) {
        uint32_t ka, kb;
        asm("s_mov_b32 %0, 0xbf80" : "=s"(ka));
        asm("s_mov_b32 %0, 0xbf800000" : "=s"(kb));
#pragma unroll
        for (int n = 0; n < N; ++n) {
            w[n] = cvt_pk(a, b);
            if (n + 1 < N) {
                const bf16x2_t h = __builtin_bit_cast(bf16x2_t, w[n]);
                a = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2_t, ka), a, false);
                b = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2_t, kb), b, false);
            }
        }
    }
    template <int N>
    static __device__ __forceinline__ void split(const f32x8& x, Terms<Frag, N>& o) {
        uint32_t w[4][N];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_pair<N>(x[2 * i], x[2 * i + 1], w[i]);
#pragma unroll
        for (int n = 0; n < N; ++n)
            o.t[n] = __builtin_bit_cast(bf16x8, u32x4{w[0][n], w[1][n], w[2][n], w[3][n]});
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
    // Whether one of two packed values is infinite or no number: an exponent of all
    // ones carries into the sign's place.
    static __device__ __forceinline__ uint32_t bad(uint32_t v) {
        return ((v & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
    }
};

// fp32 inputs: chunks of 32 tokens on the fp32 matrix cores.  A lane's 8 elements of
// a 32-deep contraction go in one at a time: the contraction's order is free.
struct F32 {
    typedef float T;
    static constexpr bool is_bf16 = false;
    static constexpr int C = 32;
    static constexpr int EP = 4;
    static constexpr int NO = 1, NS = 1;
    typedef f32x8 Frag;
    template <int N>
    static __device__ __forceinline__ void split(const f32x8& x, Terms<Frag, N>& o) {
        o.t[0] = x;
    }
    static __device__ __forceinline__ f32x8 widen(const Frag& f) { return f; }
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = mfma_f32(a[i], b[i], c);
        return c;
    }
    static __device__ __forceinline__ uint32_t bad(uint32_t v) {
        return ((v & 0x7fffffffu) + 0x00800000u) & 0x80000000u;
    }
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// LDS by byte addresses, so that a base, a constant and an exclusive or make an operand's
// address in one instruction.
template <class V> __device__ __forceinline__ V lds_get(uint32_t at, uint32_t more) {
    typedef __attribute__((address_space(3))) const char lds_c;
    typedef __attribute__((address_space(3))) const V lds_v;
    return *(lds_v*)((lds_c*)(uintptr_t)at + more);
}

__device__ __forceinline__ s16x4 lds_tr16_at(uint32_t at, uint32_t more) {
    typedef __attribute__((address_space(3))) char lds_c;
    typedef __attribute__((address_space(3))) s16x4 lds_v;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v*)((lds_c*)(uintptr_t)at + more));
}

template <class V> __device__ __forceinline__ void lds_set(uint32_t at, uint32_t more, const V& v) {
    typedef __attribute__((address_space(3))) char lds_c;
    typedef __attribute__((address_space(3))) V lds_v;
    *(lds_v*)((lds_c*)(uintptr_t)at + more) = v;
}

__device__ __forceinline__ uint32_t lds_at(const void* p) {
    typedef __attribute__((address_space(3))) const char lds_c;
    return (uint32_t)(uintptr_t)(lds_c*)p;
}

// A tile of rows of W elements in LDS, and where a lane (g = lane / 16, m = lane % 16)
// finds its operands in it.
template <class P, int W, int KIND> struct Tile {
    typedef typename P::T T;
    static constexpr int PPR = W / P::EP;           // 16-byte pieces per row
    static __device__ __forceinline__ int swizzle(int row) {
        if constexpr (!P::is_bf16) return row & (PPR - 1) & 15;
        else if constexpr (KIND == ROWS) return row & (PPR - 1);
        else if constexpr (PPR == 16) return ((row & 3) << 1) | (row & 8);
        else return (row & 2) | ((row & 8) >> 1);
    }
    static __device__ __forceinline__ int piece(int row, int c) {
        return row * W + (c ^ swizzle(row)) * P::EP;
    }
    static __device__ __forceinline__ int at(int row, int col) {
        return piece(row, col / P::EP) + col % P::EP;
    }

    // A lane's first element of an operand, as an LDS address in bytes; the others
    // differ in bits that the swizzle leaves alone or flips alike, so they are one
    // exclusive or away (tiles lie at multiples of 512 bytes), and rows a constant.
    // fresh() keeps the compiler from holding all of them in registers over a loop.

    // Elements 32 k + 8 g .. + 7 of row 16 i + m (the swizzle repeats every 16 rows).
    struct Rows {
        uint32_t o, a;
        __device__ __forceinline__ void init(int lane) {
            const int g = lane >> 4, m = lane & 15;
            o = piece(m, 8 / P::EP * g) * (uint32_t)sizeof(T);
        }
        __device__ __forceinline__ void of(const T* t) { a = o + lds_at(t); }
        __device__ __forceinline__ void fresh() { asm volatile("" : "+v"(a)); }
        __device__ __forceinline__ typename P::Frag get(int i, int k) const {
            const uint32_t row = 16 * i * W * (uint32_t)sizeof(T);
            if constexpr (P::is_bf16) {
                return __builtin_bit_cast(bf16x8, lds_get<u32x4>(a ^ (64 * k), row));
            } else {
                const f32x4 x = lds_get<f32x4>(a ^ (128 * k), row);
                const f32x4 y = lds_get<f32x4>(a ^ (128 * k + 16), row);
                return f32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
            }
        }
    };

    // Rows 32 j + 8 g .. + 7 of column 16 u + m; `column` 16 more.
    struct Cols {
        static constexpr int N = P::is_bf16 ? 2 : 8;
        uint32_t o[N], a[N];
        __device__ __forceinline__ void init(int lane, int column = 0) {
            const int g = lane >> 4, m = lane & 15;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                // bf16: lane 4 r + c of a group points at 4 columns of row r (lds_tr16)
                const int e = P::is_bf16 ? at(8 * g + (m >> 2) + 4 * i, 4 * (m & 3))
                                         : at(8 * g + i, m);
                o[i] = (e ^ (16 * column)) * (uint32_t)sizeof(T);
            }
        }
        __device__ __forceinline__ void of(const T* t) {
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = o[i] + lds_at(t);
        }
        __device__ __forceinline__ typename P::Frag get(int j, int u) const {
            const uint32_t row = 32 * j * W * (uint32_t)sizeof(T);
            const uint32_t f = 16 * u * (uint32_t)sizeof(T);
            if constexpr (P::is_bf16) {
                return pair(lds_tr16_at(a[0] ^ f, row), lds_tr16_at(a[1] ^ f, row));
            } else {
                f32x8 v;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = lds_get<float>(a[i] ^ f, row);
                return v;
            }
        }
    };

    static __device__ __forceinline__ bf16x8 pair(const s16x4& a, const s16x4& b) {
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    }
};

// P (its tiles of 16 x 16 tokens on and below the diagonal, and those above it that
// share a 32-deep contraction with them, which stay 0) in LDS, 32 columns at a time:
// rows 0 .. C - 1 of columns 0 .. 31, then (bf16) rows 32 .. 63 of columns 32 .. 63.
template <class P> struct PTile {
    typedef typename P::T T;
    static constexpr int SIZE = P::is_bf16 ? 64 * 32 + 32 * 32 : 32 * 32;
    static __device__ __forceinline__ int piece(int row, int c) {
        // four pieces a row in bf16, eight in fp32
        return row * 32 + (c ^ (P::is_bf16 ? ((row & 8) ? 3 : 0) : (row & 7))) * P::EP;
    }
    // Offset of tile (i, j) beyond that of its lane.
    static constexpr int tile(int i, int j) { return j / 2 * (32 * 32) + 16 * i * 32; }
    static __device__ __forceinline__ int at(int row, int col) {
        return piece(row % 16, col % 32 / P::EP) + col % P::EP + tile(row / 16, col / 16);
    }
    // Elements 32 j + 8 g .. + 7 of row 16 i + m, as in Tile.
    struct Rows {
        static constexpr int N = P::is_bf16 ? 1 : 2;
        uint32_t a[N];
        __device__ __forceinline__ void init(int lane, const T* t) {
            const int g = lane >> 4, m = lane & 15;
#pragma unroll
            for (int i = 0; i < N; ++i)
                a[i] = lds_at(t) + piece(m, N * g + i) * (uint32_t)sizeof(T);
        }
        // of the term that lies `t` elements behind the first
        __device__ __forceinline__ typename P::Frag get(int t, int i, int j) const {
            const uint32_t at = (t + tile(i, 2 * j)) * (uint32_t)sizeof(T);
            if constexpr (P::is_bf16) {
                return __builtin_bit_cast(bf16x8, lds_get<u32x4>(a[0], at));
            } else {
                const f32x4 x = lds_get<f32x4>(a[0], at), y = lds_get<f32x4>(a[1], at);
                return f32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
            }
        }
    };
};

// The pieces of a [C, W] tile that one of 256 threads moves from memory: piece i is
// row row0 + i C / N of the chunk, 16 bytes at channel col.
template <class P, int W, int KIND> struct Stage {
    static constexpr int PPR = W / P::EP;
    static constexpr int N = P::C * PPR / 256, STEP = P::C / N;
    typedef Tile<P, W, KIND> Tl;
    u32x4 w[N];
    int row0, col;
    uint32_t to;                    // bytes into the tile
    bool wide, narrow;              // whether the tensor has these channels, all of W
    uint32_t off;                   // bytes from a whole chunk's first token
    __device__ __forceinline__ void init(int tid, int width, int64_t st, bool back) {
        row0 = tid / PPR;
        const int c = tid % PPR * P::EP;
        wide = c < width;
        narrow = width < W;
        col = wide ? c : 0;
        to = Tl::piece(row0, tid % PPR) * (uint32_t)sizeof(typename P::T);
        const uint32_t sb = (uint32_t)(st * sizeof(typename P::T));
        off = (back ? P::C - 1 - row0 : row0) * sb + col * (uint32_t)sizeof(typename P::T);
    }
    // `chunk`: the first token's first channel.  Rows from len on are loaded as the
    // last one, and cleared by put.
    __device__ __forceinline__ void load(const char* chunk, int64_t st, int len, bool back) {
        const char* at[N];
        uint32_t o[N];
        const int64_t pass = (back ? -STEP : STEP) * st * (int)sizeof(typename P::T);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            at[i] = chunk + i * pass;
            o[i] = off;
        }
        if (len < P::C) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = row0 + i * STEP < len ? row0 + i * STEP : len - 1;
                at[i] = chunk;
                o[i] = (uint32_t)((back ? len - 1 - r : r) * st + col) *
                       (uint32_t)sizeof(typename P::T);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (P::is_bf16)
                w[i] = *reinterpret_cast<const u32x4_e2*>(at[i] + o[i]);
            else
                w[i] = *reinterpret_cast<const u32x4_e4*>(at[i] + o[i]);
        }
    }
    __device__ __forceinline__ void put(typename P::T* tile, int len) {
        if (narrow || len < P::C) {
            const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (!wide || row0 + i * STEP >= len) w[i] = zero;
        }
        const uint32_t at = lds_at(tile) + to;
#pragma unroll
        for (int i = 0; i < N; ++i)
            lds_set(at ^ flip(i), i * STEP * W * (uint32_t)sizeof(typename P::T), w[i]);
    }
    // What row0 + i STEP changes in the swizzle (which repeats every 16 rows).
    static constexpr uint32_t flip(int i) {
        if constexpr (STEP % 16 == 0) return 0;
        else return (Tl::swizzle(STEP) * (i & 1)) * 16;
    }
    // Whether an element is infinite or no number.
    __device__ __forceinline__ bool bad() const {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) any |= P::bad(w[i][j]);
        return any != 0;
    }
};

// Where a workgroup works: the (sequence, head, segment) groups go round the 8 XCDs,
// and all jobs and channel blocks of one group stay on one, whose L2 they share.
struct Place {
    int64_t b, h, seg;
    int job, zb;
};

// Workgroup id, where each has `width` channels of z.
__device__ __forceinline__ bool place(const LaChain& a, uint32_t id, int width, Place& o) {
    uint32_t nz[3], per = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        nz[j] = j < a.njobs ? (a.job[j].zd + width - 1) / width : 0;
        per += nz[j];
    }
    // a grid, and so every count here, is below 2^24
    const uint32_t H = (uint32_t)a.H, B = (uint32_t)a.B;
    const uint32_t row = id / 8, grp = row / per * 8 + id % 8, bh = grp / H;
    uint32_t k = row % per;
    o.seg = bh / B;
    if (o.seg >= a.nseg) return false;
    o.job = 0;
    while (k >= nz[o.job]) k -= nz[o.job++];
    o.zb = k;
    o.h = grp % H;
    o.b = bh % B;
    return true;
}

__device__ __forceinline__ const void* head_base(const LaTensor& t, int64_t b, int64_t h,
                                                 size_t elem) {
    const int64_t at = (uint32_t)h / (uint32_t)t.share;
    return static_cast<const char*>(t.p) + (b * t.sb + at * t.sh) * elem;
}

// Log decay that the state goes through before token t is added, as it lies in
// memory (a value that is waited for only where it is used), and in base 2.
__device__ __forceinline__ float decay_of(const LaChain& a, int64_t b, int64_t h, int64_t t) {
    if (!a.g || t >= a.T) return 0.f;
    return a.g_head ? a.g[h] : a.g[(b * a.T + t) * a.H + h];
}

__device__ __forceinline__ double base2(float g) {
    return (double)(g < kLeast ? kLeast : g) * 1.4426950408889634;
}

// Inclusive sums over the 64 lanes of a wave in 64 bits: rows of 16 by row_shr 1, 2, 4,
// 8, then across rows by row_bcast 15 and 31.
template <int CTRL, int ROW_MASK = 0xF> __device__ __forceinline__ double dpp_mov64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROW_MASK,
                                                              0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL,
                                                              ROW_MASK, 0xF, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ double wave_scan64(double x) {
    x += dpp_mov64<0x111>(x);
    x += dpp_mov64<0x112>(x);
    x += dpp_mov64<0x114>(x);
    x += dpp_mov64<0x118>(x);
    x += dpp_mov64<0x142, 0xA>(x);
    x += dpp_mov64<0x143, 0xC>(x);
    return x;
}

// The value of one lane, for all.
__device__ __forceinline__ double lane64(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

}  // namespace la
}  // namespace gdr
