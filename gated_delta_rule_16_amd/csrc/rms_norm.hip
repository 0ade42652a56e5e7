// gdr_rms_norm_fwd / _quant / _bwd: RMS norm over rows of C channels,
//
//   h = x (+ r, stored),  y = h rstd w,  rstd = 1 / sqrt(mean h^2 + eps),
//
// y in fp32 or bf16, or in 8 bits with scale max |y| / largest per row or group; and
// its reverse mode, with n = h rstd and dn = dy w:
//
//   dh = rstd (dn - n mean(dn n)) (+ dr),   dw = sum_rows dy n.
//
// Bound by HBM: one pass over each tensor, a row in registers between its
// reductions: one wave per row up to 2048 channels (1024 backward), four up to 8192,
// eight up to 16384; longer rows are walked once per reduction (from L2).  32768 x 2048
// bf16 with a residual: e4m3 in groups of 128 97 us (4.8 TB/s; int8 101), backward 107 (5.0 TB/s);
// forward 8192 x 2048 25 (5.4 TB/s).
#include "block_launch.h"
#include "linear_launch.h"
#include "norm_rows.h"

namespace gdr {

namespace {

typedef uint32_t u32x2_e1 __attribute__((ext_vector_type(2), aligned(1)));

// What an 8-bit output stores: the largest magnitude, and a value's byte.
constexpr float kE4m3Max = 448.f, kInt8Max = 127.f;

template <int Q8> __device__ __forceinline__ float largest() {
    return Q8 == 1 ? kE4m3Max : kInt8Max;
}

// Eight values as bytes (e4m3: v_cvt_pk_fp8_f32, round to nearest even, NaN kept).
template <int Q8> __device__ __forceinline__ u32x2_e1 pack8(const float (&f)[E]) {
    u32x2_e1 o;
    if constexpr (Q8 == 1) {
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], b, true);
        o.x = (uint32_t)a;
        o.y = (uint32_t)b;
    } else {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float r = fminf(fmaxf(__builtin_rintf(f[e]), -kInt8Max), kInt8Max);
            w[e / 4] |= ((uint32_t)(int)r & 0xffu) << (8 * (e % 4));
        }
        o.x = w[0];
        o.y = w[1];
    }
    return o;
}

// Channels [0, valid) of eight as bytes.
template <int Q8>
__device__ __forceinline__ void store8(void* base, int64_t off, const float (&f)[E], int valid) {
    const u32x2_e1 w = pack8<Q8>(f);
    uint8_t* p = static_cast<uint8_t*>(base) + off;
    if (valid >= E) {
        *reinterpret_cast<u32x2_e1*>(p) = w;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < valid) p[e] = (uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e % 4)));
    }
}

// Magnitudes compare as their bits, where no number is above all numbers: the
// largest of some is no number if one of them is none.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL> __device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
    return umax(x, __float_as_uint(dpp_mov<CTRL>(__uint_as_float(x))));
}

// Over the lanes of a group of `group` channels (32, 64 or 128: 4, 8 or 16 lanes).
__device__ __forceinline__ uint32_t group_max(uint32_t x, int64_t group) {
    x = dpp_max<0xB1>(x);
    x = dpp_max<0x4E>(x);
    if (group >= 64) x = dpp_max<0x141>(x);
    if (group >= 128) x = dpp_max<0x140>(x);
    return x;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = group_max(x, 128);
    x = umax(x, (uint32_t)__shfl_xor((int)x, 16, 64));
    x = umax(x, (uint32_t)__shfl_xor((int)x, 32, 64));
    return x;
}

// Scale of a group whose largest magnitude is m.
template <int Q8> __device__ __forceinline__ float scale_of(uint32_t m) {
    const float s = __uint_as_float(m) / largest<Q8>();
    return s < 1.17549435e-38f ? 0.f : s;
}

// Values over their scale: quotients, since products with a rounded reciprocal fall on
// the other side of a code's border where the quotient lies on it (32768 x 2048: 97 us,
// 94 with products).
__device__ __forceinline__ void unscale(float (&f)[E], float s) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = s == 0.f ? 0.f : f[e] / s;
}

// 1 / sqrt(mean square + eps).  An infinite sum of squares gives 0.
__device__ __forceinline__ float rstd_of(const RmsArgs& a, float ss) {
    return 1.f / sqrtf(ss * (1.f / (float)a.C) + a.eps);
}

// NV groups of 8 channels per thread, WR waves per row (1: four rows to a
// workgroup).  Q8: 0 fp32 or bf16 out, 1 e4m3, 2 int8.
template <int NV, int WR, bool BF16, int RES, bool RAG, int Q8>
__global__ __launch_bounds__(threads(WR)) void rms_fwd_kernel(RmsArgs a) {
    __shared__ float red[8];
    __shared__ uint32_t redm[8];
    constexpr bool WG = WR > 1;
    constexpr int NT = 64 * WR;
    const int id = WG ? threadIdx.x : (threadIdx.x & 63);
    const int64_t row = WG ? blockIdx.x
                           : (int64_t)blockIdx.x * 4 +
                                 __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= a.R) return;           // a whole wave (WG: never)
    float h[NV][E];
    float s = 0.f;
    SumIn<BF16, RES, false> in[NV];
    int64_t at[NV];
    int v[NV], twice[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        at[k] = (int64_t)(k * NT + id) * E;
        v[k] = own_group<RAG>(at[k], a.C, twice[k]);
        in[k].load(a, row, at[k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        in[k].sum(h[k]);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (!RAG || e >= twice[k]) s = __builtin_fmaf(h[k][e], h[k][e], s);
    }
    const float rstd = rstd_of(a, row_total<WR>(s, red));
    uint32_t most = 0;
    uint32_t gmost[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        // after the sum's barrier: h may be the residual, which a moved group
        // of another wave has read by now
        if constexpr (RES != 0) row_store<E, false>(a.h, row * a.C + at[k], RES == 1, h[k], v[k]);
        float w[E];
        if (a.w) param_load<E>(w, a.w + at[k], v[k]);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            h[k][e] *= rstd;
            if (a.w) h[k][e] *= w[e];
            m = umax(m, v[k] > 0 ? magnitude(h[k][e]) : 0u);
        }
        if constexpr (Q8 == 0) {
            row_store<E, false>(a.y, row * a.C + at[k], a.out_bf16, h[k], v[k]);
        } else {
            gmost[k] = m;
            most = umax(most, m);
        }
    }
    if constexpr (Q8 != 0) {
        float scale;
        const bool whole = a.group == a.C;
        if (whole) {
            most = wave_max(most);
            if constexpr (WG) {
                if ((threadIdx.x & 63) == 0) redm[threadIdx.x >> 6] = most;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < WR; ++i) most = umax(most, redm[i]);
            }
            scale = scale_of<Q8>(most);
            if (id == 0) a.scales[row] = scale;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!whole) {
                scale = scale_of<Q8>(group_max(gmost[k], a.group));
                if (v[k] > 0 && at[k] % a.group == 0)
                    a.scales[row * (a.C / a.group) + at[k] / a.group] = scale;
            }
            unscale(h[k], scale);
            if (v[k] > 0) store8<Q8>(a.y, row * a.C + at[k], h[k], E);
        }
    }
}

// Rows not held in registers: read once per reduction (with a residual the stored
// sum is what the later walks read; each thread its own channels).
template <bool BF16, int RES, int Q8>
__global__ __launch_bounds__(256) void rms_fwd_long_kernel(RmsArgs a) {
    __shared__ float red[4];
    __shared__ uint32_t redm[4];
    const int64_t row = blockIdx.x;
    const int64_t step = 256 * E;
    float s = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
        SumIn<BF16, RES, true> in;
        float h[E];
        in.load(a, row, c, left(a.C, c));
        in.sum(h);
        if constexpr (RES != 0) row_store<E>(a.h, row * a.C + c, RES == 1, h, left(a.C, c));
#pragma unroll
        for (int e = 0; e < E; ++e) s = __builtin_fmaf(h[e], h[e], s);
    }
    const void* src = RES ? a.h : a.x;
    constexpr bool sbf = RES ? RES == 1 : BF16;
    const int64_t so = row * (RES ? a.C : a.xr);
    const float rstd = rstd_of(a, row_total<4>(s, red));
    auto normed = [&](int64_t c, float (&h)[E]) {
        Row<E, sbf, true> r;
        float w[E];
        const int v = left(a.C, c);
        r.load(src, so + c, v);
        r.unpack(h);
        if (a.w) param_load<E>(w, a.w + c, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            h[e] *= rstd;
            if (a.w) h[e] *= w[e];
        }
        return v;
    };
    if constexpr (Q8 == 0) {
        for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
            float h[E];
            const int v = normed(c, h);
            row_store<E>(a.y, row * a.C + c, a.out_bf16, h, v);
        }
    } else {
        const bool whole = a.group == a.C;
        float scale = 0.f;
        if (whole) {
            uint32_t most = 0;
            for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
                float h[E];
                const int v = normed(c, h);
#pragma unroll
                for (int e = 0; e < E; ++e) most = umax(most, e < v ? magnitude(h[e]) : 0u);
            }
            most = wave_max(most);
            if ((threadIdx.x & 63) == 0) redm[threadIdx.x >> 6] = most;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) most = umax(most, redm[i]);
            scale = scale_of<Q8>(most);
            if (threadIdx.x == 0) a.scales[row] = scale;
        }
        for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
            float h[E];
            const int v = normed(c, h);
            if (!whole) {           // C is a multiple of the group, so its lanes are all here
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) m = umax(m, magnitude(h[e]));
                scale = scale_of<Q8>(group_max(m, a.group));
                if (c % a.group == 0) a.scales[row * (a.C / a.group) + c / a.group] = scale;
            }
            unscale(h, scale);
            store8<Q8>(a.y, row * a.C + c, h, v);
        }
    }
}

// Backward: a persistent grid walks the rows; dw stays in registers over all rows of
// a wave (WG: of the workgroup) and leaves as one partial row [C] per workgroup.
template <int NV, int WR, bool BF16, bool DY16, bool G16, bool RAG>
__global__ __launch_bounds__(threads(WR)) void rms_bwd_kernel(RmsBwdArgs a) {
    constexpr bool WG = WR > 1, AHEAD = WR < 8;
    __shared__ float red[2][2][8];
    __shared__ float join[WG ? 1 : 3 * 64 * (E + 1)];
    constexpr int NT = 64 * WR;
    const int id = WG ? threadIdx.x : (threadIdx.x & 63);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float dw[NV][E];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[k][e] = 0.f;
    const float inv = 1.f / (float)a.C;
    const int64_t stride = (int64_t)gridDim.x * (WG ? 1 : 4);
    int64_t at[NV];
    int v[NV], twice[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        at[k] = (int64_t)(k * NT + id) * E;
        v[k] = own_group<RAG>(at[k], a.C, twice[k]);
    }
    Row<E, BF16, false> rh[NV];
    Row<E, DY16, false> rd[NV];
    Row<E, G16, false> rr[NV];
    // the weights of a thread's channels: kept where they are few
    constexpr bool KEEP = NV <= 2;
    float kept[KEEP ? NV : 1][E];
    auto load_weights = [&](float (&w)[E], int k) {
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = 1.f;
        if (a.w) param_load<E>(w, a.w + at[k], v[k]);
    };
    auto weights = [&](float (&w)[E], int k) {
        if constexpr (KEEP) {
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = kept[k][e];
        } else {
            load_weights(w, k);
        }
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int k = 0; k < NV; ++k) load_weights(kept[k], k);
    }
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            rh[k].load(a.x, row * a.xr + at[k], v[k]);
            rd[k].load(a.dy, row * a.yr + at[k], v[k]);
            rr[k].load(a.dres, row * a.rr + at[k], a.dres ? v[k] : 0);
        }
    };
    int64_t row = WG ? blockIdx.x : (int64_t)blockIdx.x * 4 + wv;
    if (AHEAD && row < a.R) fetch(row);
    for (int turn = 0; row < a.R; row += stride, turn ^= 1) {
        if (!AHEAD) fetch(row);
        float h[NV][E], d[NV][E], q[NV][E];
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[E];
            weights(w, k);
            rh[k].unpack(h[k]);
            rd[k].unpack(d[k]);
            rr[k].unpack(q[k]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (RAG && e < twice[k]) continue;
                ss = __builtin_fmaf(h[k][e], h[k][e], ss);
                sd = __builtin_fmaf(d[k][e] * w[e], h[k][e], sd);
            }
        }
        // the next row's loads land while this one is worked on
        if (AHEAD && row + stride < a.R) fetch(row + stride);
        // both sums with one barrier; its slots are written again two rows on
        ss = wave_sum(ss);
        sd = wave_sum(sd);
        if constexpr (WG) {
            if ((threadIdx.x & 63) == 0) {
                red[turn][0][threadIdx.x >> 6] = ss;
                red[turn][1][threadIdx.x >> 6] = sd;
            }
            __syncthreads();
            ss = join_waves<WR>(red[turn][0]);
            sd = join_waves<WR>(red[turn][1]);
        }
        const float rstd = 1.f / sqrtf(ss * inv + a.eps);
        const float m2 = sd * inv * rstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[E], out[E];
            weights(w, k);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float n = h[k][e] * rstd;
                dw[k][e] = __builtin_fmaf(d[k][e], n, dw[k][e]);
                out[e] = rstd * (d[k][e] * w[e] - n * m2);
                out[e] += q[k][e];
            }
            row_store<E, false>(a.dx, row * a.C + at[k], G16, out, v[k]);
        }
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * a.C;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if constexpr (!WG) {
            // the four waves hold the same channels: join them, group by group
            if (k > 0) __syncthreads();
            if (wv > 0) {
                float* p = join + ((wv - 1) * 64 + id) * (E + 1);
#pragma unroll
                for (int e = 0; e < E; ++e) p[e] = dw[k][e];
            }
            __syncthreads();
            if (wv > 0) continue;
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const float* p = join + (q * 64 + id) * (E + 1);
#pragma unroll
                for (int e = 0; e < E; ++e) dw[k][e] += p[e];
            }
        }
        row_store<E, false>(part, at[k], false, dw[k], v[k]);
    }
}

// Rows not held in registers: dx first, a workgroup per row; the column sums by a
// second kernel that walks the rows with each row's rstd.
template <bool BF16, bool DY16, bool G16>
__global__ __launch_bounds__(256) void rms_bwd_long_kernel(RmsBwdArgs a, float* stats) {
    __shared__ float red[2][4];
    const int64_t row = blockIdx.x;
    const int64_t step = 256 * E;
    const float inv = 1.f / (float)a.C;
    float ss = 0.f, sd = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
        Row<E, BF16, true> rh;
        Row<E, DY16, true> rd;
        float h[E], d[E], w[E];
        const int v = left(a.C, c);
        rh.load(a.x, row * a.xr + c, v);
        rd.load(a.dy, row * a.yr + c, v);
        if (a.w) param_load<E>(w, a.w + c, v);
        rh.unpack(h);
        rd.unpack(d);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float dn = a.w ? d[e] * w[e] : d[e];
            ss = __builtin_fmaf(h[e], h[e], ss);
            sd = __builtin_fmaf(dn, h[e], sd);
        }
    }
    const float rstd = 1.f / sqrtf(row_total<4>(ss, red[0]) * inv + a.eps);
    const float m2 = row_total<4>(sd, red[1]) * inv * rstd;
    if (stats && threadIdx.x == 0) stats[row] = rstd;
    for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
        Row<E, BF16, true> rh;
        Row<E, DY16, true> rd;
        Row<E, G16, true> rr;
        float h[E], d[E], w[E], q[E];
        const int v = left(a.C, c);
        rh.load(a.x, row * a.xr + c, v);
        rd.load(a.dy, row * a.yr + c, v);
        rr.load(a.dres, row * a.rr + c, a.dres ? v : 0);
        if (a.w) param_load<E>(w, a.w + c, v);
        rh.unpack(h);
        rd.unpack(d);
        rr.unpack(q);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float dn = a.w ? d[e] * w[e] : d[e];
            h[e] = rstd * (dn - h[e] * rstd * m2);
            h[e] += q[e];
        }
        row_store<E>(a.dx, row * a.C + c, G16, h, v);
    }
}

// Column sums of the long rows: a wave owns 64 groups of 8 channels, a workgroup's
// four waves take every fourth of its rows.
template <bool BF16, bool DY16>
__global__ __launch_bounds__(256) void rms_dw_long_kernel(RmsBwdArgs a, const float* stats,
                                                          int64_t ncb, int64_t nrow) {
    __shared__ float join[3 * 64 * (E + 1)];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t cb = blockIdx.x % ncb, slot = blockIdx.x / ncb;
    const int64_t c = (cb * 64 + lane) * E;
    const int v = left(a.C, c);
    float dw[E];
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = 0.f;
    if (v > 0)
        for (int64_t row = slot * 4 + wv; row < a.R; row += nrow * 4) {
            Row<E, BF16, true> rh;
            Row<E, DY16, true> rd;
            float h[E], d[E];
            rh.load(a.x, row * a.xr + c, v);
            rd.load(a.dy, row * a.yr + c, v);
            rh.unpack(h);
            rd.unpack(d);
            const float rstd = stats[row];
#pragma unroll
            for (int e = 0; e < E; ++e) dw[e] = __builtin_fmaf(d[e], h[e] * rstd, dw[e]);
        }
    if (wv > 0) {
        float* p = join + ((wv - 1) * 64 + lane) * (E + 1);
#pragma unroll
        for (int e = 0; e < E; ++e) p[e] = dw[e];
    }
    __syncthreads();
    if (wv > 0 || v == 0) return;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        const float* p = join + (q * 64 + lane) * (E + 1);
#pragma unroll
        for (int e = 0; e < E; ++e) dw[e] += p[e];
    }
    row_store<E>(a.part + slot * a.C, c, false, dw, v);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t WG_MAX = 16384;

// Whether a row is held in registers: not beyond WG_MAX channels, nor under one
// group of them.
bool fits(int64_t C) { return C >= E && C <= WG_MAX; }

// Whether a workgroup of eight waves takes a row.
bool wide(int64_t C) { return fits(C) && C > 8192; }

// Workgroups of the backward (= partial rows), as many as fill the chip evenly.
int64_t bwd_rows(int64_t R, int64_t C) {
    if (!fits(C)) {
        const int64_t cap = cdiv(2048, cdiv(C, 64 * E));
        const int64_t n = cdiv(R, 16);
        return n < cap ? n : cap;
    }
    const int64_t per = C <= 1024 ? 4 : 1, most = cdiv(R, per), want = cdiv(R, 16 * per);
    const int64_t n = want < 256 ? 256 : want > 1024 ? 1024 : want;
    return n < most ? n : most;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int NV, int WR, bool BF16, int RES, int Q8>
void fwd_r(const RmsArgs& a, dim3 grid) {
    if (a.C % E)
        hipLaunchKernelGGL((rms_fwd_kernel<NV, WR, BF16, RES, true, Q8>), grid, dim3(threads(WR)),
                           0, a.stream, a);
    else
        hipLaunchKernelGGL((rms_fwd_kernel<NV, WR, BF16, RES, false, Q8>), grid, dim3(threads(WR)),
                           0, a.stream, a);
}

template <bool BF16, int RES, int Q8>
void fwd_q(const RmsArgs& a) {
    const int64_t C = a.C;
    const dim3 wave((unsigned)cdiv(a.R, 4)), wg((unsigned)a.R);
    if (!fits(C))
        hipLaunchKernelGGL((rms_fwd_long_kernel<BF16, RES, Q8>), wg, dim3(256), 0, a.stream, a);
    else if (C <= 512) fwd_r<1, 1, BF16, RES, Q8>(a, wave);
    else if (C <= 1024) fwd_r<2, 1, BF16, RES, Q8>(a, wave);
    else if (C <= 2048) fwd_r<4, 1, BF16, RES, Q8>(a, wave);
    else if (C <= 4096) fwd_r<2, 4, BF16, RES, Q8>(a, wg);
    else if (!wide(C)) fwd_r<4, 4, BF16, RES, Q8>(a, wg);
    else fwd_r<4, 8, BF16, RES, Q8>(a, wg);
}

template <bool BF16, int RES>
void fwd_t(const RmsArgs& a) {
    if (a.q8 == 0) fwd_q<BF16, RES, 0>(a);
    else if (a.q8 == 1) fwd_q<BF16, RES, 1>(a);
    else fwd_q<BF16, RES, 2>(a);
}

template <bool BF16>
void fwd_b(const RmsArgs& a) {
    if (!a.res) fwd_t<BF16, 0>(a);
    else if (a.res_bf16) fwd_t<BF16, 1>(a);
    else fwd_t<BF16, 2>(a);
}

template <int NV, int WR, bool BF16, bool DY16, bool G16>
void bwd_r(const RmsBwdArgs& a, dim3 grid) {
    if (a.C % E)
        hipLaunchKernelGGL((rms_bwd_kernel<NV, WR, BF16, DY16, G16, true>), grid,
                           dim3(threads(WR)), 0, a.stream, a);
    else
        hipLaunchKernelGGL((rms_bwd_kernel<NV, WR, BF16, DY16, G16, false>), grid,
                           dim3(threads(WR)), 0, a.stream, a);
}

template <bool BF16, bool DY16, bool G16>
void bwd_t(const RmsBwdArgs& a) {
    const int64_t C = a.C, nrow = bwd_rows(a.R, C);
    const dim3 grid((unsigned)nrow);
    if (fits(C)) {
        if (C <= 512) bwd_r<1, 1, BF16, DY16, G16>(a, grid);
        else if (C <= 1024) bwd_r<2, 1, BF16, DY16, G16>(a, grid);
        else if (C <= 2048) bwd_r<1, 4, BF16, DY16, G16>(a, grid);
        else if (C <= 4096) bwd_r<2, 4, BF16, DY16, G16>(a, grid);
        else if (!wide(C)) bwd_r<4, 4, BF16, DY16, G16>(a, grid);
        else bwd_r<4, 8, BF16, DY16, G16>(a, grid);
    } else {
        const int64_t ncb = cdiv(C, 64 * E);
        float* stats = a.part ? reinterpret_cast<float*>(reinterpret_cast<char*>(a.part) +
                                up256(sizeof(float) * (size_t)(nrow * C))) : nullptr;
        hipLaunchKernelGGL((rms_bwd_long_kernel<BF16, DY16, G16>), dim3((unsigned)a.R), dim3(256),
                           0, a.stream, a, stats);
        if (a.part)
            hipLaunchKernelGGL((rms_dw_long_kernel<BF16, DY16>), dim3((unsigned)(ncb * nrow)),
                               dim3(256), 0, a.stream, a, stats, ncb, nrow);
    }
}

template <bool BF16>
void bwd_b(const RmsBwdArgs& a) {
    if (a.dy_bf16) {
        if (a.grad_bf16) bwd_t<BF16, true, true>(a);
        else bwd_t<BF16, true, false>(a);
    } else {
        if (a.grad_bf16) bwd_t<BF16, false, true>(a);
        else bwd_t<BF16, false, false>(a);
    }
}

}  // namespace

double rms_work_items(int64_t R, int64_t C) {
    return (double)R * (wide(C) ? threads(8) : threads(1));
}

size_t rms_bwd_workspace_bytes(int64_t R, int64_t C) {
    size_t n = up256(sizeof(float) * (size_t)(bwd_rows(R, C) * C));
    if (!fits(C)) n += sizeof(float) * (size_t)R;
    return n;
}

hipError_t launch_rms_fwd(const RmsArgs& a) {
    if (a.in_bf16) fwd_b<true>(a);
    else fwd_b<false>(a);
    return hipGetLastError();
}

hipError_t launch_rms_bwd(const RmsBwdArgs& a) {
    if (a.in_bf16) bwd_b<true>(a);
    else bwd_b<false>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    return launch_sum_partials(a.part, bwd_rows(a.R, a.C), a.C, a.dw, a.C, nullptr, a.stream);
}

}  // namespace gdr
