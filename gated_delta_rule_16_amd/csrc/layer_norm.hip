// gdr_layer_norm_fwd / _bwd: the block's pre-norm over rows of C channels,
//
//   h = x (+ r, stored), mu = mean h, v = mean (h - mu)^2,
//   y = (h - mu) / sqrt(v + eps) * w + b,
//
// and its reverse mode, with n = (h - mu) rstd and dn = dy w:
//
//   dh = rstd (dn - mean dn - n mean(dn n)) (+ dr),  dw = sum_rows dy n,  db = sum_rows dy.
//
// Bound by HBM: one pass over each tensor.  A row is held in registers
// between its two reductions (mean, then the centred squares, so there is no
// cancellation of mean squares): one wave per row up to 2048 channels (1024
// backward), with no barrier; a workgroup of four waves per row up to 8192, of
// eight up to 16384; beyond that the workgroup walks the row again (from L2) for
// each reduction.
// 32768 rows of 2048 in bf16 with the residual stream: forward 99 us (5.4
// TB/s), backward 107 us (5.0 TB/s; a copy reaches 4.9 to 5.4 on the same card).
#include "block_launch.h"
#include "norm_rows.h"

namespace gdr {

namespace {

// Three sums at once.
template <int WR>
__device__ __forceinline__ void row_totals(float (&x)[3], float (*red)[8]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) x[i] = wave_sum(x[i]);
    if constexpr (WR > 1) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < 3; ++i) red[i][threadIdx.x >> 6] = x[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) x[i] = join_waves<WR>(red[i]);
    }
}

// NV groups of 8 channels per thread, WR waves per row (1: four rows to a
// workgroup).
template <int NV, int WR, bool BF16, int RES, bool RAG>
__global__ __launch_bounds__(threads(WR)) void norm_fwd_kernel(NormArgs a) {
    __shared__ float red[2][8];
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
        for (int e = 0; e < E; ++e) s += !RAG || e >= twice[k] ? h[k][e] : 0.f;
    }
    const float inv = 1.f / (float)a.C;
    const float mu = row_total<WR>(s, red[0]) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        // after the sum's barrier: h may be the residual, which a moved group
        // of another wave has read by now
        if constexpr (RES != 0) row_store<E, false>(a.h, row * a.C + at[k], RES == 1, h[k], v[k]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            h[k][e] -= mu;
            if (v[k] > 0 && (!RAG || e >= twice[k])) s = __builtin_fmaf(h[k][e], h[k][e], s);
        }
    }
    const float rstd = 1.f / sqrtf(row_total<WR>(s, red[1]) * inv + a.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        float w[E], b[E];
        if (a.w) param_load<E>(w, a.w + at[k], v[k]);
        if (a.b) param_load<E>(b, a.b + at[k], v[k]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float y = h[k][e] * rstd;
            if (a.w) y *= w[e];
            if (a.b) y += b[e];
            h[k][e] = y;
        }
        row_store<E, false>(a.y, row * a.C + at[k], a.out_bf16, h[k], v[k]);
    }
}

// Rows too long for registers: the row is read once per reduction.  With a
// residual the stored sum is what the later walks read (each thread its own
// channels, so no barrier is needed between its store and its loads).
template <bool BF16, int RES>
__global__ __launch_bounds__(256) void norm_fwd_long_kernel(NormArgs a) {
    __shared__ float red[2][4];
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
        for (int e = 0; e < E; ++e) s += h[e];
    }
    const void* src = RES ? a.h : a.x;
    constexpr bool sbf = RES ? RES == 1 : BF16;
    const int64_t so = row * (RES ? a.C : a.xr);
    const float inv = 1.f / (float)a.C;
    const float mu = row_total<4>(s, red[0]) * inv;
    s = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
        Row<E, sbf, true> r;
        float h[E];
        const int v = left(a.C, c);
        r.load(src, so + c, v);
        r.unpack(h);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < v) s = __builtin_fmaf(h[e] - mu, h[e] - mu, s);
    }
    const float rstd = 1.f / sqrtf(row_total<4>(s, red[1]) * inv + a.eps);
    for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
        Row<E, sbf, true> r;
        float h[E], w[E], b[E];
        const int v = left(a.C, c);
        r.load(src, so + c, v);
        r.unpack(h);
        if (a.w) param_load<E>(w, a.w + c, v);
        if (a.b) param_load<E>(b, a.b + c, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float y = (h[e] - mu) * rstd;
            if (a.w) y *= w[e];
            if (a.b) y += b[e];
            h[e] = y;
        }
        row_store<E>(a.y, row * a.C + c, a.out_bf16, h, v);
    }
}

// Backward: a persistent grid walks the rows; dw and db stay in registers
// over all rows of a wave (WG: of the workgroup) and leave as one partial row
// [2 C] per workgroup.  From 1024 channels on the workgroup shares a row: a
// wave that holds 2048 channels of three tensors, their sums and the next row
// leaves one wave per SIMD (32768 rows of 2048 in bf16: 126 us without the next
// row's loads, 152 with them, 111 shared; 107 with the weights kept in registers
// too).  Eight waves leave no registers for the next row's loads (2113 rows of
// 15613 in fp32: 250 us with them, 137 without).
template <int NV, int WR, bool BF16, bool DY16, bool G16, bool RAG>
__global__ __launch_bounds__(threads(WR)) void norm_bwd_kernel(NormBwdArgs a) {
    constexpr bool WG = WR > 1, AHEAD = WR < 8;
    __shared__ float red[4][8];
    __shared__ float join[WG ? 1 : 3 * 64 * (2 * E + 1)];
    constexpr int NT = 64 * WR;
    const int id = WG ? threadIdx.x : (threadIdx.x & 63);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float dw[NV][E], db[NV][E];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[k][e] = db[k][e] = 0.f;
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
    for (; row < a.R; row += stride) {
        if (!AHEAD) fetch(row);
        float h[NV][E], d[NV][E], q[NV][E];
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            rh[k].unpack(h[k]);
            rd[k].unpack(d[k]);
            rr[k].unpack(q[k]);
#pragma unroll
            for (int e = 0; e < E; ++e) s += !RAG || e >= twice[k] ? h[k][e] : 0.f;
        }
        // the next row's loads land while this one is worked on
        if (AHEAD && row + stride < a.R) fetch(row + stride);
        const float mu = row_total<WR>(s, red[0]) * inv;
        float sums[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[E];
            weights(w, k);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                h[k][e] = v[k] > 0 ? h[k][e] - mu : 0.f;
                if (RAG && e < twice[k]) continue;
                sums[0] = __builtin_fmaf(h[k][e], h[k][e], sums[0]);
                const float dn = d[k][e] * w[e];
                sums[1] += dn;
                sums[2] = __builtin_fmaf(dn, h[k][e], sums[2]);
            }
        }
        row_totals<WR>(sums, red + 1);
        const float rstd = 1.f / sqrtf(sums[0] * inv + a.eps);
        const float m1 = sums[1] * inv, m2 = sums[2] * inv * rstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[E], out[E];
            weights(w, k);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float n = h[k][e] * rstd;
                const float dn = d[k][e] * w[e];
                dw[k][e] = __builtin_fmaf(d[k][e], n, dw[k][e]);
                db[k][e] += d[k][e];
                out[e] = rstd * (dn - m1 - n * m2);
                out[e] += q[k][e];
            }
            row_store<E, false>(a.dx, row * a.C + at[k], G16, out, v[k]);
        }
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.C;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if constexpr (!WG) {
            // the four waves hold the same channels: join them, group by group
            if (k > 0) __syncthreads();
            if (wv > 0) {
                float* p = join + ((wv - 1) * 64 + id) * (2 * E + 1);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    p[e] = dw[k][e];
                    p[E + e] = db[k][e];
                }
            }
            __syncthreads();
            if (wv > 0) continue;
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const float* p = join + (q * 64 + id) * (2 * E + 1);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    dw[k][e] += p[e];
                    db[k][e] += p[E + e];
                }
            }
        }
        row_store<E, false>(part, at[k], false, dw[k], v[k]);
        row_store<E, false>(part, a.C + at[k], false, db[k], v[k]);
    }
}

// Rows too long for registers: dx first, a workgroup per row; the column sums
// by a second kernel that walks the rows with each row's mean and rstd.
template <bool BF16, bool DY16, bool G16>
__global__ __launch_bounds__(256) void norm_bwd_long_kernel(NormBwdArgs a, float* stats) {
    __shared__ float red[4][4];
    const int64_t row = blockIdx.x;
    const int64_t step = 256 * E;
    const float inv = 1.f / (float)a.C;
    float s = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * E; c < a.C; c += step) {
        Row<E, BF16, true> r;
        float h[E];
        r.load(a.x, row * a.xr + c, left(a.C, c));
        r.unpack(h);
#pragma unroll
        for (int e = 0; e < E; ++e) s += h[e];
    }
    const float mu = row_total<4>(s, red[0]) * inv;
    s = 0.f;
    float s1 = 0.f, s2 = 0.f;
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
            const float x = e < v ? h[e] - mu : 0.f;
            const float dn = a.w ? d[e] * w[e] : d[e];
            s = __builtin_fmaf(x, x, s);
            s1 += dn;
            s2 = __builtin_fmaf(dn, x, s2);
        }
    }
    const float rstd = 1.f / sqrtf(row_total<4>(s, red[1]) * inv + a.eps);
    const float m1 = row_total<4>(s1, red[2]) * inv;
    const float m2 = row_total<4>(s2, red[3]) * inv * rstd;
    if (stats && threadIdx.x == 0) {
        stats[2 * row] = mu;
        stats[2 * row + 1] = rstd;
    }
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
            h[e] = rstd * (dn - m1 - (h[e] - mu) * rstd * m2);
            h[e] += q[e];
        }
        row_store<E>(a.dx, row * a.C + c, G16, h, v);
    }
}

// Column sums of the long rows: a wave owns 64 groups of 8 channels, a
// workgroup's four waves take every fourth of its rows.
template <bool BF16, bool DY16>
__global__ __launch_bounds__(256) void norm_dw_long_kernel(NormBwdArgs a, const float* stats,
                                                           int64_t ncb, int64_t nrow) {
    __shared__ float join[3 * 64 * (2 * E + 1)];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t cb = blockIdx.x % ncb, slot = blockIdx.x / ncb;
    const int64_t c = (cb * 64 + lane) * E;
    const int v = left(a.C, c);
    float dw[E], db[E];
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = db[e] = 0.f;
    if (v > 0)
        for (int64_t row = slot * 4 + wv; row < a.R; row += nrow * 4) {
            Row<E, BF16, true> rh;
            Row<E, DY16, true> rd;
            float h[E], d[E];
            rh.load(a.x, row * a.xr + c, v);
            rd.load(a.dy, row * a.yr + c, v);
            rh.unpack(h);
            rd.unpack(d);
            const float mu = stats[2 * row], rstd = stats[2 * row + 1];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                dw[e] = __builtin_fmaf(d[e], (h[e] - mu) * rstd, dw[e]);
                db[e] += d[e];
            }
        }
    if (wv > 0) {
        float* p = join + ((wv - 1) * 64 + lane) * (2 * E + 1);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            p[e] = dw[e];
            p[E + e] = db[e];
        }
    }
    __syncthreads();
    if (wv > 0 || v == 0) return;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        const float* p = join + (q * 64 + lane) * (2 * E + 1);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            dw[e] += p[e];
            db[e] += p[E + e];
        }
    }
    float* part = a.part + slot * 2 * a.C;
    row_store<E>(part, c, false, dw, v);
    row_store<E>(part, a.C + c, false, db, v);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t WG_MAX = 16384;

// Whether a row is held in registers: not beyond WG_MAX channels, nor under one
// group of them.
bool fits(int64_t C) { return C >= E && C <= WG_MAX; }

// Workgroups of the backward (= partial rows).
int64_t bwd_rows(int64_t R, int64_t C) {
    if (!fits(C)) {
        const int64_t cap = cdiv(2048, cdiv(C, 64 * E));
        const int64_t n = cdiv(R, 16);
        return n < cap ? n : cap;
    }
    // a wave (up to 1024 channels) or the workgroup per row.  1024 workgroups
    // fill the chip evenly, four to a compute unit (32768 rows of 2048 in bf16:
    // 111 us; 139 with 512, 152 with 1536); fewer rows take fewer, so that the
    // partials stay a small part of the traffic
    const int64_t per = C <= 1024 ? 4 : 1, most = cdiv(R, per), want = cdiv(R, 16 * per);
    const int64_t n = want < 256 ? 256 : want > 1024 ? 1024 : want;
    return n < most ? n : most;
}

// Whether a workgroup of eight waves takes a row.
bool wide(int64_t C) { return fits(C) && C > 8192; }

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int NV, int WR, bool BF16, int RES>
void fwd_r(const NormArgs& a, dim3 grid) {
    if (a.C % E)
        hipLaunchKernelGGL((norm_fwd_kernel<NV, WR, BF16, RES, true>), grid, dim3(threads(WR)), 0,
                           a.stream, a);
    else
        hipLaunchKernelGGL((norm_fwd_kernel<NV, WR, BF16, RES, false>), grid, dim3(threads(WR)), 0,
                           a.stream, a);
}

template <bool BF16, int RES>
void fwd_t(const NormArgs& a) {
    const int64_t C = a.C;
    const dim3 wave((unsigned)cdiv(a.R, 4)), wg((unsigned)a.R);
    if (!fits(C))
        hipLaunchKernelGGL((norm_fwd_long_kernel<BF16, RES>), wg, dim3(256), 0, a.stream, a);
    else if (C <= 512) fwd_r<1, 1, BF16, RES>(a, wave);
    else if (C <= 1024) fwd_r<2, 1, BF16, RES>(a, wave);
    else if (C <= 2048) fwd_r<4, 1, BF16, RES>(a, wave);
    else if (C <= 4096) fwd_r<2, 4, BF16, RES>(a, wg);
    else if (!wide(C)) fwd_r<4, 4, BF16, RES>(a, wg);
    else fwd_r<4, 8, BF16, RES>(a, wg);
}

template <bool BF16>
void fwd_b(const NormArgs& a) {
    if (!a.res) fwd_t<BF16, 0>(a);
    else if (a.res_bf16) fwd_t<BF16, 1>(a);
    else fwd_t<BF16, 2>(a);
}

template <int NV, int WR, bool BF16, bool DY16, bool G16>
void bwd_r(const NormBwdArgs& a, dim3 grid) {
    if (a.C % E)
        hipLaunchKernelGGL((norm_bwd_kernel<NV, WR, BF16, DY16, G16, true>), grid,
                           dim3(threads(WR)), 0, a.stream, a);
    else
        hipLaunchKernelGGL((norm_bwd_kernel<NV, WR, BF16, DY16, G16, false>), grid,
                           dim3(threads(WR)), 0, a.stream, a);
}

template <bool BF16, bool DY16, bool G16>
void bwd_t(const NormBwdArgs& a) {
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
                                up256(sizeof(float) * (size_t)(nrow * 2 * C))) : nullptr;
        hipLaunchKernelGGL((norm_bwd_long_kernel<BF16, DY16, G16>), dim3((unsigned)a.R), dim3(256),
                           0, a.stream, a, stats);
        if (a.part)
            hipLaunchKernelGGL((norm_dw_long_kernel<BF16, DY16>), dim3((unsigned)(ncb * nrow)),
                               dim3(256), 0, a.stream, a, stats, ncb, nrow);
    }
}

template <bool BF16>
void bwd_b(const NormBwdArgs& a) {
    if (a.dy_bf16) {
        if (a.grad_bf16) bwd_t<BF16, true, true>(a);
        else bwd_t<BF16, true, false>(a);
    } else {
        if (a.grad_bf16) bwd_t<BF16, false, true>(a);
        else bwd_t<BF16, false, false>(a);
    }
}

}  // namespace

// Work-items of the forward, a workgroup per row (or fewer: one wave up to 2048
// channels).
double norm_fwd_work_items(int64_t R, int64_t C) {
    return (double)R * (wide(C) ? threads(8) : threads(1));
}

// Workspace: the partials of dw and db [bwd_rows][2 C], and each row's mean and
// rstd where the row is not held in registers.
size_t norm_bwd_workspace_bytes(int64_t R, int64_t C) {
    size_t n = up256(sizeof(float) * (size_t)(bwd_rows(R, C) * 2 * C));
    if (!fits(C)) n += sizeof(float) * (size_t)(2 * R);
    return n;
}

hipError_t launch_norm_fwd(const NormArgs& a) {
    if (a.in_bf16) fwd_b<true>(a);
    else fwd_b<false>(a);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwdArgs& a) {
    if (a.in_bf16) bwd_b<true>(a);
    else bwd_b<false>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    return launch_sum_partials(a.part, bwd_rows(a.R, a.C), 2 * a.C, a.dw, a.C, a.db,
                               a.stream);
}

}  // namespace gdr
