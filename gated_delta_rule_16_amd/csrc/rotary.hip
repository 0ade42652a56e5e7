// gdr_rotary: the first channels of every head of q and k as pairs, turned by
// position times rate.
//
// Bound by HBM: one read and one write of every element (bf16 B8 T4096, 16 and 16 heads
// of 128: 98 us, 5.5 TB/s; a thread's own sines and cosines 143).  A workgroup takes a
// few tokens: it forms the sines and cosines of their angles once, in LDS, and its
// threads walk the heads side by side, 8 channels (in the half layout with the 8 of
// their partners) to a thread, so a wave reads consecutive memory.
#include "linear_launch.h"
#include "mfma_common.h"
#include "rows.h"

namespace gdr {

namespace {

constexpr int E = 8;
constexpr int TB = 4;       // tokens with their loads in flight at once

// sin and cos of pos f.  The angle in quarter turns is a sum of two doubles, with what
// the products pos f and (pos f) (2 / pi) round off and 2 / pi in two terms, so the
// reduction loses nothing at far positions either (three rounded products would be off
// by 2^-12 at position 2^40 and rate 1).  The rest is at most about half a quarter turn,
// where the Taylor series to x^9 and x^10 err by 2e-9.
__device__ __forceinline__ void sincos_at(double pos, double f, float& s, float& c) {
#pragma clang fp contract(off)          // t is what fma(angle, kHi, -t) says it is
    constexpr double kHi = 0x1.45f306dc9c883p-1, kLo = -0x1.6b01ec5417056p-55;     // 2 / pi
    const double angle = pos * f, t = angle * kHi;
    const double more = __builtin_fma(angle, kHi, -t) +
                        __builtin_fma(angle, kLo, __builtin_fma(pos, f, -angle) * kHi);
    const double n = __builtin_rint(t);
    const float x = (float)(((t - n) + more) * 1.5707963267948966);
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

// An item is 8 channels of a head: `turning` of its units turn (half layout: 8 pairs
// each), the others are copied.  A thread keeps its item over its tokens.
template <bool BF16, bool INTER, bool RAG>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
    constexpr int NF = INTER ? E / 2 : E;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    struct Token {
        int64_t qi, qo, ki, ko;
        double pos;
    };
    Token* const tokens = reinterpret_cast<Token*>(smem);
    float2* const turn = reinterpret_cast<float2*>(smem + a.tokens * sizeof(Token));
    const int tid = threadIdx.x, half = (int)a.rot / 2;
    const int64_t n = a.B * a.T, first = (int64_t)blockIdx.x * a.tokens;
    const int nt = (int)(n - first < a.tokens ? n - first : a.tokens);
    if (tid < nt) {
        const int64_t b = (first + tid) / a.T, t = (first + tid) % a.T;
        Token k;
        k.qi = b * a.q.ib + t * a.q.it;
        k.qo = b * a.q.ob + t * a.q.ot;
        k.ki = b * a.k.ib + t * a.k.it;
        k.ko = b * a.k.ob + t * a.k.ot;
        k.pos = (double)(a.positions ? a.positions[b * a.pos_stride + t] : a.start + t);
        tokens[tid] = k;
    }
    __syncthreads();
    for (int i = tid; i < nt * half; i += 256) {
        float s, c;
        sincos_at(tokens[i / half].pos, a.freqs[i % half], s, c);
        turn[i] = float2{c * a.scale, s * (a.inverse ? -a.scale : a.scale)};
    }
    __syncthreads();
    const int heads = (int)(a.Hq + a.Hk), items = heads * a.units;
    // fewer items than threads: several tokens side by side
    const int side = items >= 256 ? 1 : 256 / items;
    const int t0 = side > 1 ? tid / items : 0;
    if (t0 >= side) return;
    for (int item = side > 1 ? tid % items : tid; item < items; item += 256) {
        const int unit = item % a.units, h = item / a.units;
        const bool isq = h < a.Hq, turns = unit < a.turning;
        const void* const in = isq ? a.q.in : a.k.in;
        void* const out = isq ? a.q.out : a.k.out;
        const int c0 = turns ? unit * E : (int)a.rot + (unit - a.turning) * E;
        const int end = turns ? (INTER ? (int)a.rot : half) : (int)a.D;
        const int v0 = end - c0 < E ? end - c0 : E;
        const int v1 = !INTER && turns ? v0 : 0;          // partners
        const int64_t hi = (isq ? h * a.q.ih : (h - a.Hq) * a.k.ih) + c0;
        const int64_t ho = (isq ? h * a.q.oh : (h - a.Hq) * a.k.oh) + c0;
        const int f0 = INTER ? c0 / 2 : c0;
        // all loads of a few tokens before the first store (which a later load of the
        // same memory would have to wait for)
        for (int tb = t0; tb < nt; tb += TB * side) {
            Row<E, BF16, RAG> r0[TB], r1[INTER ? 1 : TB];
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                const int t = tb + i * side;
                const Token& k = tokens[t < nt ? t : tb];
                const int64_t at = (isq ? k.qi : k.ki) + hi;
                r0[i].load(in, at, t < nt ? v0 : 0);
                if constexpr (!INTER) r1[i].load(in, at + half, t < nt ? v1 : 0);
            }
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                const int t = tb + i * side;
                if (t >= nt) break;
                const int64_t at = (isq ? tokens[t].qo : tokens[t].ko) + ho;
                if (!turns) {
                    r0[i].copy_to(out, at, v0);
                    continue;
                }
                float cs[NF], sn[NF];
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    const int g = !RAG || f0 + f < half ? f0 + f : half - 1;
                    const float2 v = turn[t * half + g];
                    cs[f] = v.x;
                    sn[f] = v.y;
                }
                float x[E], y[E];
                r0[i].unpack(x);
                if constexpr (INTER) {
#pragma unroll
                    for (int f = 0; f < NF; ++f) {
                        y[2 * f] = x[2 * f] * cs[f] - x[2 * f + 1] * sn[f];
                        y[2 * f + 1] = x[2 * f] * sn[f] + x[2 * f + 1] * cs[f];
                    }
                    row_store<E, RAG>(out, at, BF16, y, v0);
                } else {
                    float w[E], z[E];
                    r1[i].unpack(w);
#pragma unroll
                    for (int f = 0; f < NF; ++f) {
                        y[f] = x[f] * cs[f] - w[f] * sn[f];
                        z[f] = x[f] * sn[f] + w[f] * cs[f];
                    }
                    row_store<E, RAG>(out, at, BF16, y, v0);
                    row_store<E, RAG>(out, at + half, BF16, z, v1);
                }
            }
        }
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <bool BF16, bool INTER> void go(const RotaryArgs& a, dim3 grid) {
    const bool whole = (INTER ? a.rot : a.rot / 2) % E == 0 && (a.D - a.rot) % E == 0;
    const size_t lds = a.tokens * (5 * 8 + 8 * (size_t)(a.rot / 2));
    if (whole)
        hipLaunchKernelGGL((rotary_kernel<BF16, INTER, false>), grid, dim3(256), lds, a.stream, a);
    else
        hipLaunchKernelGGL((rotary_kernel<BF16, INTER, true>), grid, dim3(256), lds, a.stream, a);
}

}  // namespace

// Units and tokens per workgroup of a call.  In place, what does not turn is left
// alone.
void rotary_shape(RotaryArgs& a) {
    a.turning = (int)cdiv(a.interleaved ? a.rot : a.rot / 2, E);
    const bool same = a.q.in == a.q.out && (a.Hk == 0 || a.k.in == a.k.out);
    a.units = a.turning + (same ? 0 : (int)cdiv(a.D - a.rot, E));
    // 4 items a thread (B8 T4096 bf16, heads of 128: 16 and 16 98 us, with 2 items 96,
    // with 8 100; 32 and 8 121, 135, 126), sines and cosines in 32 KB, and no fewer
    // workgroups than twice the compute units where that leaves them tokens
    int64_t n = 1024 / ((a.Hq + a.Hk) * a.units);
    const int64_t most = 4096 / (a.rot / 2), few = a.B * a.T / 512;
    if (n > most) n = most;
    if (n > few) n = few;
    if (n > 64) n = 64;
    a.tokens = (int)(n < 1 ? 1 : n);
}

double rotary_work_items(const RotaryArgs& a) {
    return ((double)a.B * (double)a.T / a.tokens + 1.0) * 256.0;
}

hipError_t launch_rotary(const RotaryArgs& a) {
    const dim3 grid((unsigned)cdiv(a.B * a.T, a.tokens));
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
