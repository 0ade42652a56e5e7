// gdr_ssm_scan_fwd and gdr_ssm_step: the selective state space scan
//
//   Delta_t = softplus(dt_t + dt_bias),
//   h_t[n] = exp(Delta_t A[n]) h_{t-1}[n] + Delta_t x_t B_t[n],
//   y_t = sum_n C_t[n] h_t[n] + D x_t   (times z_t sigmoid(z_t)),
//
// per channel, with N states each; B and C are shared by the channels of a
// group.  The decay differs per state, so no product of matrices covers a
// stretch of tokens: the scan runs on the vector ALU, one exp, two products
// and two fused adds per state and token (25 cycles per 64 of them on gfx950,
// measured), in fp32 throughout.
//
// Work split (ssm.h): rows of 16 lanes are channels, so B and C enter as row
// broadcasts.  A tile of tokens is staged in LDS by waves that do nothing else
// (Delta and Delta x once per channel, B and C as fp32), so the token loop has
// no global access; two tiles' loads are in flight.  B 8 T 4096 D 2048 N 16,
// gated, bf16: 264 us, 2.0 TB/s, with the vector ALU busy in 95% of the cycles
// (437 us where the scanning waves also staged).
//
// Few channels: the sequence is cut into segments that run side by side.  A
// first pass leaves each segment's end state from zero and the sum of its
// Delta (whose exp with A is the segment's decay); the second starts from the
// states composed of those.  It costs a second exp per state, so it is taken
// only where the channels alone leave most of the chip idle (ssm_fwd_plan).
#include <type_traits>

#include "ssm.h"

namespace gdr {

namespace {

template <int NS, int NG, bool OUT, bool BF16, bool RAG>
__global__ __launch_bounds__(64 * (NG + 4)) void ssm_fwd_kernel(SsmArgs a, int64_t nblk,
                                                                int64_t nseg, int64_t L) {
    constexpr int NP = NS * NG, CW = WC / NG;
    constexpr int EPT = 8;                            // staged channels per thread
    constexpr int TT = 256 * EPT / WC;                // tokens per tile
    constexpr int TPR = WC / EPT;                     // threads per token row
    constexpr int NQ = TT * NP / 4;                   // groups of 4 of B (and of C) per tile
    constexpr int QPT = (2 * NQ + 255) / 256;
    constexpr int KT = 16 / NS;                       // tokens per B register
    constexpr int YP = WC + 16;                       // pitch: 4 tokens' stores meet no bank twice
    __shared__ float2 dd[2][TT][WC];
    __shared__ __align__(16) float bc[2][2][TT * NP];
    __shared__ float ys[2][OUT ? TT : 1][YP];

    const int lane = threadIdx.x & 63, tid = (int)threadIdx.x - 64 * NG;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool scans = wv < NG;
    int64_t id = blockIdx.x;
    const int64_t blk = id % nblk;
    id /= nblk;
    const int64_t g = id % a.G;
    id /= a.G;
    const int64_t ns = OUT ? nseg : nseg - 1;         // the last segment's end state is not needed
    const int64_t seg = id % ns, b = id / ns;
    const int64_t Dg = a.D / a.G, cg = g * Dg;
    const int64_t c0 = first_channel<RAG>(blk, Dg);
    const int64_t t0 = seg * L, t1 = t0 + L < a.T ? t0 + L : a.T;
    const int64_t tiles = (t1 - t0 + TT - 1) / TT;

    if (scans) {
        // the lane's channel and states
        const int row = lane >> 4, n0 = NS * (row % NG);
        const int chl = wv * CW + (lane & 15) + 16 * (row / NG);
        const bool live = c0 + chl < Dg;
        const int64_t ch = cg + (live ? c0 + chl : 0);
        const int nv = live ? states_valid<NS>(a.N, n0) : 0;
        float A2[NS], h[NS];
        param_load<NS>(A2, a.A + ch * a.N + n0, nv);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            A2[j] = decay_rate(A2[j]);
            h[j] = 0.f;
        }
        const int64_t so = (b * a.D + ch) * a.N + n0;
        // hend[b][0] is h0 as the first pass copied it (the second pass must
        // not read h0: another workgroup may be writing h_final, the same
        // buffer), hend[b][s] the end of segment s - 1, segment 0 started from h0
        if (!OUT || nseg == 1) {
            if (a.h0 && seg == 0) states_load<NS>(h, a.h0 + so, nv);
            if constexpr (!OUT)
                if (seg == 0)
                    states_store<NS>(a.hend + (b * nseg * a.D + ch) * NP + n0, h, live ? NS : 0);
        } else {
            states_load<NS, false>(h, a.hend + ((b * nseg + (seg > 0)) * a.D + ch) * NP + n0, live);
            const int64_t o = (b * nseg + 1) * a.D + ch;
            compose<NS>(h, A2, a.hend + (o + a.D) * NP + n0, a.D * NP, a.sdelta + o, a.D, seg - 1,
                        live);
        }
        float sumd = 0.f;
        __syncthreads();
        for (int64_t i = 0; i < tiles; ++i) {
            const int buf = (int)(i & 1);
            const int64_t tb = t0 + i * TT;
            const int nt = t1 - tb < TT ? (int)(t1 - tb) : TT;
            auto group = [&](int tt) {
                float Bq[4 / KT], Cq[4 / KT];
                float2 d[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) d[k] = dd[buf][tt + k][chl];
#pragma unroll
                for (int k = 0; k < 4 / KT; ++k) {
                    Bq[k] = row_coef<NS, NG>(bc[buf][0], tt + k * KT, lane);
                    Cq[k] = OUT ? row_coef<NS, NG>(bc[buf][1], tt + k * KT, lane) : 0.f;
                }
                constexpr auto js = std::make_index_sequence<NS>{};
                float ea[4][NS], bx[4][NS];
                scan_terms<NS, 0 % KT>(ea[0], bx[0], A2, d[0].x, d[0].y, Bq[0 / KT], js);
                scan_terms<NS, 1 % KT>(ea[1], bx[1], A2, d[1].x, d[1].y, Bq[1 / KT], js);
                scan_terms<NS, 2 % KT>(ea[2], bx[2], A2, d[2].x, d[2].y, Bq[2 / KT], js);
                scan_terms<NS, 3 % KT>(ea[3], bx[3], A2, d[3].x, d[3].y, Bq[3 / KT], js);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int j = 0; j < NS; ++j)
                        bx[k][j] =
                            __builtin_fmaf(ea[k][j], k ? bx[k ? k - 1 : 0][j] : h[j], bx[k][j]);
                }
                if constexpr (OUT) {
                    float s[4];
                    row_dots<NS>(s, Cq, bx);
                    state_sums<NG>(s, row, &ys[buf][tt][chl], YP);
                } else {
                    sumd += (d[0].x + d[1].x) + (d[2].x + d[3].x);
                }
#pragma unroll
                for (int j = 0; j < NS; ++j) h[j] = bx[3][j];
            };
            // a token past the end moves nothing, so whole groups may run
            for (int tt = 0; tt < nt; tt += 8) {
                group(tt);
                group(tt + 4);
            }
            __syncthreads();
        }
        if constexpr (OUT) {
            if (a.h_final && seg == nseg - 1) states_store<NS>(a.h_final + so, h, nv);
        } else {
            const int64_t o = (b * nseg + seg) * a.D + ch;
            states_store<NS>(a.hend + (o + a.D) * NP + n0, h, live ? NS : 0);
            if (live && n0 == 0) a.sdelta[o] = sumd;
        }
        return;
    }

    // the other four waves: each thread's part of the staging
    const int srow = tid / TPR, sc = (tid % TPR) * EPT;
    const int sv = ssm_left(Dg, c0 + sc, EPT);
    const int64_t scg = cg + c0 + sc;
    float bias[EPT], skip[EPT];
    param_load<EPT>(bias, a.bias + scg, a.bias ? sv : 0);
    param_load<EPT>(skip, a.D_skip + scg, OUT && a.D_skip ? sv : 0);
    // addresses of the next tile to fetch: of x, dt, z, and of B or C
    using T = typename std::conditional<BF16, bf16_t, float>::type;
    const T* px = static_cast<const T*>(a.x) + b * a.xb + (t0 + srow) * a.xt + scg;
    const T* pt = static_cast<const T*>(a.dt) + b * a.dtb + (t0 + srow) * a.dtt + scg;
    const T* pz = static_cast<const T*>(a.z) + b * a.zb + (t0 + srow) * a.zt + scg;
    const T* pq[QPT];
#pragma unroll
    for (int i = 0; i < QPT; ++i) {
        const int q = tid + 256 * i, qt = (q % NQ) / (NP / 4), qn = q % (NP / 4);
        pq[i] = q >= NQ ? static_cast<const T*>(a.Cm) + b * a.cb + (t0 + qt) * a.ct
                        : static_cast<const T*>(a.Bm) + b * a.bb + (t0 + qt) * a.bt;
        pq[i] += g * a.N + quad_start<NG>(a.N, qn);
    }
    // two tiles' loads are in flight, each in its own registers
    struct Rows {
        Row<EPT, BF16, RAG> x, t, z;
        Row<4, BF16, NG == 1> q[QPT];
    } rows0, rows1;
    auto fetch = [&](int64_t i, Rows& r) {
        const int64_t tb = t0 + i * TT;
        if (tb >= t1) return;
        const int left = t1 - tb < TT ? (int)(t1 - tb) : TT;
        const int v = srow < left ? sv : 0;
        r.x.load(px, 0, v);
        r.t.load(pt, 0, v);
        px += TT * a.xt;
        pt += TT * a.dtt;
        if constexpr (OUT) {
            r.z.load(pz, 0, a.z ? v : 0);
            pz += TT * a.zt;
        }
#pragma unroll
        for (int j = 0; j < QPT; ++j) {
            const int q = tid + 256 * j;
            const bool isc = q >= NQ;
            if (isc && !OUT) continue;
            const int qt = (q % NQ) / (NP / 4), qn = q % (NP / 4);
            const int vq = q < 2 * NQ && qt < left ? quad_valid<NG>(a.N, qn) : 0;
            r.q[j].load(pq[j], 0, vq);
            pq[j] += TT * (isc ? a.ct : a.bt);
        }
    };
    // what a tile's epilogue needs: y = (sum over n + base) factor
    struct Held {
        float base[EPT], factor[EPT];
    } even, odd;
    auto stage = [&](int64_t i, const Rows& rows, Held& k) {
        const int buf = (int)(i & 1);
        // a token past the end or a channel past the group moves nothing: its
        // decay is exp(0) and it adds 0
        const int tv = t0 + i * TT + srow < t1 ? sv : 0;
        float x[EPT], r[EPT], d[EPT];
        rows.x.unpack(x);
        rows.t.unpack(r);
#pragma unroll
        for (int e = 0; e < EPT; ++e) r[e] += bias[e];
        ssm_deltas(d, r, a.softplus);
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            d[e] = (RAG ? e < tv : tv > 0) ? d[e] : 0.f;
            dd[buf][srow][sc + e] = float2{d[e], d[e] * x[e]};
        }
        if constexpr (OUT) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                k.base[e] = skip[e] * x[e];
                k.factor[e] = 1.f;
            }
            if (a.z) {
                float z[EPT];
                rows.z.unpack(z);
                ssm_gate(k.factor, z);
            }
        }
#pragma unroll
        for (int q4 = 0; q4 < QPT; ++q4) {
            const int q = tid + 256 * q4;
            if (q >= 2 * NQ || (q >= NQ && !OUT)) continue;
            float f[4];
            rows.q[q4].unpack(f);
            quad_write<NP, NG>(bc[buf][q >= NQ], q % NQ, a.N, f);
        }
    };
    int64_t oo = (b * a.T + t0 + srow) * a.D + scg;
    auto finish = [&](int64_t i, const Held& k) {
        if (t0 + i * TT + srow < t1 && sv > 0) {
            float y[EPT];
#pragma unroll
            for (int e = 0; e < EPT; ++e)
                y[e] = (ys[i & 1][srow][sc + e] + k.base[e]) * k.factor[e];
            row_store<EPT, RAG>(a.y, oo, a.out_bf16, y, sv);
        }
        oo += TT * a.D;
    };
    quad_clear<NP, 4 * TT>(&bc[0][0][0], a.N, tid);
    fetch(0, rows0);
    fetch(1, rows1);
    stage(0, rows0, even);
    fetch(2, rows0);
    __syncthreads();
    // while tile i runs: tile i + 1 is staged and tile i + 3's loads are issued;
    // then tile i goes out while tile i + 1 runs
    auto step = [&](int64_t i, const Held& now, Held& next, Rows& rows) {
        if (i + 1 < tiles) {
            stage(i + 1, rows, next);
            fetch(i + 3, rows);
        }
        __syncthreads();
        if constexpr (OUT) finish(i, now);
    };
    for (int64_t i = 0; i < tiles; i += 2) {
        step(i, even, odd, rows1);
        if (i + 1 < tiles) step(i + 1, odd, even, rows0);
    }
}

// One decode token: every lane streams its 4 states once; bound by the
// state's HBM traffic (8 bytes per state against ~6 operations): 256 sequences
// of D 2048 N 16 take 17.7 us, 4.0 TB/s.
// A workgroup takes 256 / LPC channels of one sequence.
template <int LPC, bool BF16>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmArgs a, uint32_t nblk) {
    const uint32_t blk = blockIdx.x % nblk;
    const int64_t b = blockIdx.x / nblk;
    const int ng = threadIdx.x % LPC;
    const uint32_t c = blk * (256 / LPC) + threadIdx.x / LPC;
    const bool live = c < (uint32_t)a.D;
    const int64_t ch = live ? c : 0;
    const int nv = live ? states_valid<4>(a.N, 4 * ng) : 0;
    float h[4], A4[4], B4[4], C4[4], x[1], r[1], z[1];
    const int64_t so = (b * a.D + ch) * a.N + 4 * ng;
    states_load<4>(h, a.h0 + so, nv);
    param_load<4>(A4, a.A + ch * a.N + 4 * ng, nv);
    const int64_t g = a.G == 1 ? 0 : (uint32_t)ch / (uint32_t)(a.D / a.G);
    Row<4, BF16, true> rb, rc;
    Row<1, BF16, false> rx, rt, rz;
    rb.load(a.Bm, b * a.bb + g * a.N + 4 * ng, nv);
    rc.load(a.Cm, b * a.cb + g * a.N + 4 * ng, nv);
    rx.load(a.x, b * a.xb + ch, live);
    rt.load(a.dt, b * a.dtb + ch, live);
    rz.load(a.z, b * a.zb + ch, live && a.z);
    const float bias = a.bias ? a.bias[ch] : 0.f, skip = a.D_skip ? a.D_skip[ch] : 0.f;
    rx.unpack(x);
    rt.unpack(r);
    rb.unpack(B4);
    rc.unpack(C4);
    const float d = ssm_delta(r[0] + bias, a.softplus);
    const float dx = d * x[0];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * decay_rate(A4[j])), h[j], dx * B4[j]);
        s = __builtin_fmaf(C4[j], h[j], s);
    }
    states_store<4>(a.h_final + so, h, nv);
    if constexpr (LPC >= 2) s += xor_lane<1>(s);
    if constexpr (LPC >= 4) s += xor_lane<2>(s);
    if constexpr (LPC >= 8) s += xor_lane<4>(s);
    if constexpr (LPC >= 16) s += xor_lane<8>(s);
    if (live && ng == 0) {
        float y[1] = {__builtin_fmaf(skip, x[0], s)};
        if (a.z) {
            rz.unpack(z);
            y[0] *= z[0] * sigmoid(z[0]);
        }
        row_store<1>(a.y, b * a.D + ch, a.out_bf16, y, 1);
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int NS, int NG, bool BF16, bool RAG>
hipError_t launch_fwd_r(const SsmArgs& a, const SsmPlan& p) {
    const int64_t wgs = a.B * a.G * p.nblk;
    const dim3 threads(64 * (NG + 4));
    if (p.nseg > 1) {
        hipLaunchKernelGGL((ssm_fwd_kernel<NS, NG, false, BF16, RAG>),
                           dim3((unsigned)(wgs * (p.nseg - 1))), threads, 0, a.stream, a, p.nblk,
                           p.nseg, p.L);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((ssm_fwd_kernel<NS, NG, true, BF16, RAG>), dim3((unsigned)(wgs * p.nseg)),
                       threads, 0, a.stream, a, p.nblk, p.nseg, p.L);
    return hipGetLastError();
}

template <int NS, int NG>
hipError_t launch_fwd_t(const SsmArgs& a, const SsmPlan& p) {
    const int64_t Dg = a.D / a.G;
    // a moved block reads states that another one also writes back: not where
    // h0's buffer is h_final's
    const bool rag =
        Dg % 8 != 0 && (Dg < WC || (p.nseg == 1 && a.h_final && a.h_final == a.h0));
    if (a.in_bf16)
        return rag ? launch_fwd_r<NS, NG, true, true>(a, p)
                   : launch_fwd_r<NS, NG, true, false>(a, p);
    return rag ? launch_fwd_r<NS, NG, false, true>(a, p)
               : launch_fwd_r<NS, NG, false, false>(a, p);
}

template <int LPC>
hipError_t launch_step_t(const SsmArgs& a) {
    const int64_t nblk = cdiv(a.D * LPC, 256);
    const dim3 grid((unsigned)(a.B * nblk));
    if (a.in_bf16)
        hipLaunchKernelGGL((ssm_step_kernel<LPC, true>), grid, dim3(256), 0, a.stream, a,
                           (uint32_t)nblk);
    else
        hipLaunchKernelGGL((ssm_step_kernel<LPC, false>), grid, dim3(256), 0, a.stream, a,
                           (uint32_t)nblk);
    return hipGetLastError();
}

}  // namespace

static int ssm_lanes(int64_t N) {
    int l = 1;
    while (4 * l < N) l *= 2;
    return l;
}

int64_t ssm_padded_states(int64_t N) {
    int64_t n = 4;
    while (n < N) n *= 2;
    return n;
}

// A segment costs 0.1 us at the head of every other one, and a token 0.05 us:
// about sqrt(T / 2) segments balance the two (B 1 T 32768 D 16 N 16 forward: 50 us
// with 128, 71 with 64, 73 with 512; backward 111, 172, 185).  At least 64 tokens.
int64_t ssm_most_segments(int64_t T) {
    const int64_t n = (T + 63) / 64;
    int64_t r = 1;
    while (r < n && r < 512 && 2 * (r + 1) * (r + 1) <= T) ++r;
    return r;
}

// Segments of the forward.  One when the channels give 192 workgroups, three
// quarters of one per compute unit; below that enough for two per compute unit
// (B 1 T 32768 D 2048 N 16: 417 us with 512 workgroups, 454 with 256, 556 with
// 384, 885 with 128).
SsmPlan ssm_fwd_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    SsmPlan p;
    p.nblk = cdiv(D / G, 64);
    const int64_t wgs = B * G * p.nblk;
    int64_t n = 1;
    if (wgs < 192) n = 512 / wgs;
    const int64_t most = ssm_most_segments(T);
    if (n > most) n = most;
    if (n < 1) n = 1;
    p.L = cdiv(cdiv(T, n), 32) * 32;
    p.nseg = T > 0 ? cdiv(T, p.L) : 1;
    return p;
}

// Workspace of the forward with nseg > 1: the states at segment starts as
// above [B, nseg, D, N padded], then the sums of Delta [B, nseg, D].
size_t ssm_fwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    const SsmPlan p = ssm_fwd_plan(B, T, D, G, N);
    return p.nseg > 1 ? sizeof(float) * (size_t)(B * p.nseg * D * (ssm_padded_states(N) + 1)) : 0;
}

hipError_t launch_ssm_fwd(SsmArgs a, float* ws) {
    const SsmPlan p = ssm_fwd_plan(a.B, a.T, a.D, a.G, a.N);
    a.hend = ws;
    a.sdelta = ws ? ws + a.B * p.nseg * a.D * ssm_padded_states(a.N) : nullptr;
    if (a.N <= 4) return launch_fwd_t<4, 1>(a, p);
    if (a.N <= 8) return launch_fwd_t<4, 2>(a, p);
    if (a.N <= 16) return launch_fwd_t<4, 4>(a, p);
    if (a.N <= 32) return launch_fwd_t<8, 4>(a, p);
    return launch_fwd_t<16, 4>(a, p);
}

int64_t ssm_step_workgroups(int64_t B, int64_t D, int64_t N) {
    return B * cdiv(D * ssm_lanes(N), 256);
}

hipError_t launch_ssm_step(const SsmArgs& a) {
    switch (ssm_lanes(a.N)) {
        case 1: return launch_step_t<1>(a);
        case 2: return launch_step_t<2>(a);
        case 4: return launch_step_t<4>(a);
        case 8: return launch_step_t<8>(a);
        default: return launch_step_t<16>(a);
    }
}

}  // namespace gdr
