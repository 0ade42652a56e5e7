// gdr_rotary: the first channels of every head of q and k as pairs, turned by
// position times rate.
//
// Bound by HBM: one read and one write of every element.  A thread takes 8 channels
// (and, in the half layout, the 8 of their partners) of one token, forms the 8 (4)
// angles' sine and cosine once, and walks several heads with them.
#include "linear_launch.h"
#include "mfma_common.h"
#include "rows.h"

namespace gdr {

namespace {

constexpr int E = 8;

// sin and cos of t quarter turns.  The reduction is in 64 bits; the rest is at most
// half a quarter turn, where the Taylor series to x^9 and x^10 err by 2e-9.
__device__ __forceinline__ void sincos_quarters(double t, float& s, float& c) {
    const double n = __builtin_rint(t);
    const float x = (float)((t - n) * 1.5707963267948966);
    const int k = (int)(n - 4.0 * __builtin_rint(n * 0.25)) & 3;
    const float z = x * x;
    float p = 2.7557319224e-6f;
    p = __builtin_fmaf(p, z, -1.9841269841e-4f);
    p = __builtin_fmaf(p, z, 8.3333333333e-3f);
    p = __builtin_fmaf(p, z, -1.6666666667e-1f);
    const float sn = __builtin_fmaf(p * z, x, x);
    float r = -2.7557319224e-7f;
    r = __builtin_fmaf(r, z, 2.4801587302e-5f);
    r = __builtin_fmaf(r, z, -1.3888888889e-3f);
    r = __builtin_fmaf(r, z, 4.1666666667e-2f);
    r = __builtin_fmaf(r, z, -0.5f);
    const float cs = __builtin_fmaf(r, z, 1.f);
    const float a = (k & 1) ? cs : sn, b = (k & 1) ? sn : cs;
    s = (k & 2) ? -a : a;
    c = (k == 1 || k == 2) ? -b : b;
}

// Threads: head group outermost, then tokens, then units of 8 channels: first those
// that turn (half layout: 8 pairs each), then those that are copied.
template <bool BF16, bool INTER, bool RAG>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per = a.B * a.T * a.units;
    if (id >= per * a.groups) return;
    const int unit = (int)(id % a.units);
    const int64_t tok = id / a.units % (a.B * a.T);
    const int64_t b = tok / a.T, t = tok % a.T;
    const int h0 = (int)(id / per) * a.hper;
    int h1 = h0 + a.hper;
    if (h1 > a.Hq + a.Hk) h1 = (int)(a.Hq + a.Hk);

    const bool turns = unit < a.turning;
    const int half = (int)a.rot / 2;
    const int c0 = turns ? unit * E : (int)a.rot + (unit - a.turning) * E;
    const int end = turns ? (INTER ? (int)a.rot : half) : (int)a.D;
    const int v0 = end - c0 < E ? end - c0 : E;
    const int v1 = !INTER && turns ? v0 : 0;          // partners
    constexpr int NF = INTER ? E / 2 : E;
    float sn[NF], cs[NF];
    if (turns) {
        const int64_t pos = a.positions ? a.positions[b * a.pos_stride + t] : a.start + t;
        const double p = (double)pos * 0.6366197723675814;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int i = (INTER ? c0 / 2 : c0) + f;
            sincos_quarters(p * (i < half ? a.freqs[i] : 0.0), sn[f], cs[f]);
            sn[f] *= a.inverse ? -a.scale : a.scale;
            cs[f] *= a.scale;
        }
    }
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const bool isq = h < a.Hq;
        const RotarySide& s = isq ? a.q : a.k;
        const int64_t hh = isq ? h : h - a.Hq;
        const int64_t in = b * s.ib + t * s.it + hh * s.ih + c0;
        const int64_t out = b * s.ob + t * s.ot + hh * s.oh + c0;
        Row<E, BF16, RAG> r0, r1;
        r0.load(s.in, in, v0);
        r1.load(s.in, in + half, v1);
        if (!turns) {
            r0.copy_to(s.out, out, v0);
            continue;
        }
        float x[E], y[E];
        r0.unpack(x);
        if constexpr (INTER) {
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                y[2 * f] = x[2 * f] * cs[f] - x[2 * f + 1] * sn[f];
                y[2 * f + 1] = x[2 * f] * sn[f] + x[2 * f + 1] * cs[f];
            }
            row_store<E, RAG>(s.out, out, BF16, y, v0);
        } else {
            float w[E], z[E];
            r1.unpack(w);
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                y[f] = x[f] * cs[f] - w[f] * sn[f];
                z[f] = x[f] * sn[f] + w[f] * cs[f];
            }
            row_store<E, RAG>(s.out, out, BF16, y, v0);
            row_store<E, RAG>(s.out, out + half, BF16, z, v1);
        }
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <bool BF16, bool INTER> void go(const RotaryArgs& a, dim3 grid) {
    const bool whole = (INTER ? a.rot : a.rot / 2) % E == 0 && (a.D - a.rot) % E == 0;
    if (whole) hipLaunchKernelGGL((rotary_kernel<BF16, INTER, false>), grid, dim3(256), 0, a.stream, a);
    else hipLaunchKernelGGL((rotary_kernel<BF16, INTER, true>), grid, dim3(256), 0, a.stream, a);
}

}  // namespace

// Units and head groups of a call.  In place, what does not turn is left alone.
void rotary_shape(RotaryArgs& a) {
    a.turning = (int)cdiv(a.interleaved ? a.rot : a.rot / 2, E);
    const bool same = a.q.in == a.q.out && (a.Hk == 0 || a.k.in == a.k.out);
    a.units = a.turning + (same ? 0 : (int)cdiv(a.D - a.rot, E));
    const int64_t heads = a.Hq + a.Hk, threads = a.B * a.T * a.units;
    int64_t hper = 16;
    while (hper > 1 && threads * cdiv(heads, hper) < 65536) hper /= 2;
    a.hper = (int)hper;
    a.groups = cdiv(heads, hper);
}

double rotary_work_items(const RotaryArgs& a) {
    return (double)a.B * (double)a.T * a.units * (double)a.groups + 256.0;
}

hipError_t launch_rotary(const RotaryArgs& a) {
    const dim3 grid((unsigned)cdiv(a.B * a.T * a.units * a.groups, 256));
    if (a.bf16) {
        if (a.interleaved) go<true, true>(a, grid);
        else go<true, false>(a, grid);
    } else {
        if (a.interleaved) go<false, true>(a, grid);
        else go<false, false>(a, grid);
    }
    return hipGetLastError();
}

}  // namespace gdr
