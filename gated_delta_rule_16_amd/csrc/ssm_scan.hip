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
// Work split: the four lanes of a channel at N = 16 hold 4 states each, which
// fills the chip at 16384 channels and costs 2 adds per token for the sum over n.
// A tile of tokens is staged in LDS by the whole workgroup (Delta and Delta x
// once per channel, B and C as fp32), so the token loop has no global access;
// the next tile's loads are issued before it and land during it.
//
// Few channels: the sequence is cut into segments that run side by side.  A
// first pass leaves each segment's end state from zero and the sum of its
// Delta (whose exp with A is the segment's decay); the second starts from the
// states composed of those.  It costs a second exp per state, so it is taken
// only where the channels alone leave most of the chip idle (ssm_fwd_segs).
#include "ssm.h"

namespace gdr {

namespace {

template <int LPC, bool OUT>
__global__ __launch_bounds__(256) void ssm_fwd_kernel(SsmArgs a, int64_t nblk, int64_t nseg,
                                                      int64_t L) {
    constexpr int WC = 256 / LPC;
    constexpr int TT = 8 * LPC < 32 ? 8 * LPC : 32;   // tokens per tile
    constexpr int EPT = TT * WC / 256;                // staged channels per thread
    constexpr int TPR = WC / EPT;                     // threads per token row
    constexpr int NQ = TT * LPC;                      // groups of 4 of B (and of C) per tile
    constexpr int QPT = (2 * NQ + 255) / 256;
    constexpr int YP = WC + 16;                       // pitch: 4 tokens' stores meet no bank twice
    __shared__ float2 dd[TT][WC];
    __shared__ float4 bc[TT][2][LPC];
    __shared__ float ys[OUT ? TT : 1][YP];

    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    int64_t id = blockIdx.x;
    const int64_t blk = id % nblk;
    id /= nblk;
    const int64_t g = id % a.G;
    id /= a.G;
    const int64_t ns = OUT ? nseg : nseg - 1;         // the last segment's end state is not needed
    const int64_t seg = id % ns, b = id / ns;
    const int64_t Dg = a.D / a.G, c0 = blk * WC, cg = g * Dg;
    const int64_t t0 = seg * L, t1 = t0 + L < a.T ? t0 + L : a.T;

    // the lane's channel and states
    const int ng = lane % LPC, chl = wv * (64 / LPC) + lane / LPC;
    const bool live = c0 + chl < Dg;
    const int64_t ch = cg + (live ? c0 + chl : 0);
    const int nv = live ? ssm_states(a.N, ng) : 0;
    float A2[4], h[4] = {0.f, 0.f, 0.f, 0.f};
    param_load<4>(A2, a.A + ch * a.N + 4 * ng, nv);
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[j] *= kLog2e;
    const int64_t so = (b * a.D + ch) * a.N + 4 * ng;
    // hend[b][0] is h0 as the first pass copied it (the second pass must not
    // read h0: another workgroup may be writing h_final, the same buffer),
    // hend[b][s] the end of segment s - 1, segment 0 started from h0
    if (!OUT || nseg == 1) {
        if (a.h0 && seg == 0) state_load(h, a.h0 + so, nv);
        if constexpr (!OUT)
            if (seg == 0) state_store(a.hend + (b * nseg * a.D + ch) * a.N + 4 * ng, h, nv);
    } else {
        state_load(h, a.hend + ((b * nseg + (seg > 0)) * a.D + ch) * a.N + 4 * ng, nv);
        for (int64_t s = 1; s < seg; ++s) {
            const int64_t o = (b * nseg + s) * a.D + ch;
            float e[4];
            state_load(e, a.hend + (o + a.D) * a.N + 4 * ng, nv);
            const float sd = live ? a.sdelta[o] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(A2[j] * sd), h[j], e[j]);
        }
    }

    // the thread's part of the staging
    const int srow = tid / TPR, sc = (tid % TPR) * EPT;
    const int sv = ssm_left(Dg, c0 + sc, EPT);
    const int64_t scg = cg + c0 + sc;
    float bias[EPT], skip[EPT];
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
        bias[e] = a.bias && e < sv ? a.bias[scg + e] : 0.f;
        skip[e] = OUT && a.D_skip && e < sv ? a.D_skip[scg + e] : 0.f;
    }
    RawRow<EPT> rx, rt, rz;
    RawRow<4> rq[QPT];
    auto fetch = [&](int64_t tb) {
        const int64_t t = tb + srow;
        const int v = t < t1 ? sv : 0;
        row_load<EPT>(rx, a.x, v ? b * a.xb + t * a.xt + scg : 0, a.in_bf16, v);
        row_load<EPT>(rt, a.dt, v ? b * a.dtb + t * a.dtt + scg : 0, a.in_bf16, v);
        if (OUT && a.z) row_load<EPT>(rz, a.z, v ? b * a.zb + t * a.zt + scg : 0, a.in_bf16, v);
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int q = tid + 256 * i;
            const bool isc = q >= NQ;
            if (isc && !OUT) continue;
            const int qt = (q % NQ) / LPC, qn = q % LPC;
            const int64_t tq = tb + qt;
            const int vq = q < 2 * NQ && tq < t1 ? ssm_states(a.N, qn) : 0;
            row_load<4>(rq[i], isc ? a.Cm : a.Bm,
                        vq ? (isc ? b * a.cb + tq * a.ct : b * a.bb + tq * a.bt) + g * a.N + 4 * qn
                           : 0,
                        a.in_bf16, vq);
        }
    };
    fetch(t0);
    float sumd = 0.f;
    for (int64_t tb = t0; tb < t1; tb += TT) {
        const int64_t t = tb + srow;
        const bool tok = t < t1;
        float x[EPT], z[EPT];
        row_unpack<EPT>(x, rx, a.in_bf16);
        if (OUT && a.z) row_unpack<EPT>(z, rz, a.in_bf16);
        {
            float r[EPT];
            row_unpack<EPT>(r, rt, a.in_bf16);
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                // a token past the end or a channel past the group moves nothing:
                // its decay is exp(0) and it adds 0
                float d = ssm_delta(r[e] + bias[e], a.softplus);
                d = tok && e < sv ? d : 0.f;
                dd[srow][sc + e] = float2{d, d * x[e]};
            }
        }
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int q = tid + 256 * i;
            const bool isc = q >= NQ;
            if (q >= 2 * NQ || (isc && !OUT)) continue;
            float f[4];
            row_unpack<4>(f, rq[i], a.in_bf16);
            bc[(q % NQ) / LPC][isc][q % LPC] = float4{f[0], f[1], f[2], f[3]};
        }
        __syncthreads();
        if (tb + TT < t1) fetch(tb + TT);
        const int nt = t1 - tb < TT ? (int)(t1 - tb) : TT;
        for (int tt = 0; tt < nt; tt += 4) {
            float s[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 d = dd[tt + k][chl];
                const float4 B4 = bc[tt + k][0][ng];
                const float Bv[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d.x * A2[j]), h[j], d.y * Bv[j]);
                if constexpr (OUT) {
                    const float4 C4 = bc[tt + k][1][ng];
                    s[k] = __builtin_fmaf(C4.w, h[3], __builtin_fmaf(C4.z, h[2],
                                          __builtin_fmaf(C4.y, h[1], C4.x * h[0])));
                } else {
                    sumd += d.x;
                }
            }
            if constexpr (OUT) channel_sums<LPC>(s, ng, &ys[tt][chl], YP);
        }
        __syncthreads();
        if constexpr (OUT) {
            if (tok && sv > 0) {
                float y[EPT];
#pragma unroll
                for (int e = 0; e < EPT; ++e) {
                    y[e] = __builtin_fmaf(skip[e], x[e], ys[srow][sc + e]);
                    if (a.z) y[e] *= z[e] * sigmoid(z[e]);
                }
                row_store<EPT>(a.y, (b * a.T + t) * a.D + scg, a.out_bf16, y, sv);
            }
        }
    }
    if constexpr (OUT) {
        if (a.h_final && seg == nseg - 1) state_store(a.h_final + so, h, nv);
    } else {
        const int64_t o = (b * nseg + seg) * a.D + ch;
        state_store(a.hend + (o + a.D) * a.N + 4 * ng, h, nv);
        if (live && ng == 0) a.sdelta[o] = sumd;
    }
}

// One decode token: every lane streams its 4 states once; bound by the
// state's HBM traffic (8 bytes per state against ~6 operations).
template <int LPC>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmArgs a) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int ng = (int)(id % LPC);
    const int64_t bc = id / LPC;
    const bool live = bc < a.B * a.D;
    const int64_t b = live ? bc / a.D : 0, ch = live ? bc % a.D : 0;
    const int nv = live ? ssm_states(a.N, ng) : 0;
    float h[4], A4[4], B4[4], C4[4];
    const int64_t so = (b * a.D + ch) * a.N + 4 * ng;
    state_load(h, a.h0 + so, nv);
    param_load<4>(A4, a.A + ch * a.N + 4 * ng, nv);
    const int64_t g = ch / (a.D / a.G);
    RawRow<4> rb, rc;
    RawRow<1> rx, rt, rz;
    row_load<4>(rb, a.Bm, b * a.bb + g * a.N + 4 * ng, a.in_bf16, nv);
    row_load<4>(rc, a.Cm, b * a.cb + g * a.N + 4 * ng, a.in_bf16, nv);
    row_load<1>(rx, a.x, b * a.xb + ch, a.in_bf16, live);
    row_load<1>(rt, a.dt, b * a.dtb + ch, a.in_bf16, live);
    if (a.z) row_load<1>(rz, a.z, b * a.zb + ch, a.in_bf16, live);
    float x[1], r[1], z[1];
    row_unpack<1>(x, rx, a.in_bf16);
    row_unpack<1>(r, rt, a.in_bf16);
    row_unpack<4>(B4, rb, a.in_bf16);
    row_unpack<4>(C4, rc, a.in_bf16);
    const float d = ssm_delta(r[0] + (a.bias ? a.bias[ch] : 0.f), a.softplus);
    const float dx = d * x[0];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * (A4[j] * kLog2e)), h[j], dx * B4[j]);
        s = __builtin_fmaf(C4[j], h[j], s);
    }
    state_store(a.h_final + so, h, nv);
    if constexpr (LPC >= 2) s += xor_lane<1>(s);
    if constexpr (LPC >= 4) s += xor_lane<2>(s);
    if constexpr (LPC >= 8) s += xor_lane<4>(s);
    if constexpr (LPC >= 16) s += xor_lane<8>(s);
    if (live && ng == 0) {
        float y[1] = {a.D_skip ? __builtin_fmaf(a.D_skip[ch], x[0], s) : s};
        if (a.z) {
            row_unpack<1>(z, rz, a.in_bf16);
            y[0] *= z[0] * sigmoid(z[0]);
        }
        row_store<1>(a.y, b * a.D + ch, a.out_bf16, y, 1);
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int LPC>
hipError_t launch_fwd_t(const SsmArgs& a, const SsmPlan& p) {
    if (p.nseg > 1) {
        hipLaunchKernelGGL((ssm_fwd_kernel<LPC, false>),
                           dim3((unsigned)(a.B * a.G * p.nblk * (p.nseg - 1))), dim3(256), 0,
                           a.stream, a, p.nblk, p.nseg, p.L);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((ssm_fwd_kernel<LPC, true>), dim3((unsigned)(a.B * a.G * p.nblk * p.nseg)),
                       dim3(256), 0, a.stream, a, p.nblk, p.nseg, p.L);
    return hipGetLastError();
}

template <int LPC>
hipError_t launch_step_t(const SsmArgs& a) {
    hipLaunchKernelGGL((ssm_step_kernel<LPC>), dim3((unsigned)cdiv(a.B * a.D * LPC, 256)),
                       dim3(256), 0, a.stream, a);
    return hipGetLastError();
}

}  // namespace

int ssm_lanes(int64_t N) {
    int l = 1;
    while (4 * l < N) l *= 2;
    return l;
}

// Segments of the forward.  One when the channels fill the chip: 768 waves,
// three quarters of one per SIMD.  Below that enough segments for two waves
// per SIMD, of at least 64 tokens.
SsmPlan ssm_fwd_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    SsmPlan p;
    p.lpc = ssm_lanes(N);
    p.nblk = cdiv(D / G, 256 / p.lpc);
    const int64_t waves = 4 * B * G * p.nblk;
    int64_t n = 1;
    if (waves < 768) n = cdiv(2048, waves);
    const int64_t most = cdiv(T, 64);
    if (n > most) n = most;
    if (n < 1) n = 1;
    p.L = cdiv(cdiv(T, n), 32) * 32;
    p.nseg = T > 0 ? cdiv(T, p.L) : 1;
    return p;
}

// Workspace of the forward with nseg > 1: the states at segment starts as
// above [B, nseg, D, N], then the sums of Delta [B, nseg, D].
size_t ssm_fwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    const SsmPlan p = ssm_fwd_plan(B, T, D, G, N);
    return p.nseg > 1 ? sizeof(float) * (size_t)(B * p.nseg * D * (N + 1)) : 0;
}

hipError_t launch_ssm_fwd(SsmArgs a, float* ws) {
    const SsmPlan p = ssm_fwd_plan(a.B, a.T, a.D, a.G, a.N);
    a.hend = ws;
    a.sdelta = ws ? ws + a.B * p.nseg * a.D * a.N : nullptr;
    switch (p.lpc) {
        case 1: return launch_fwd_t<1>(a, p);
        case 2: return launch_fwd_t<2>(a, p);
        case 4: return launch_fwd_t<4>(a, p);
        case 8: return launch_fwd_t<8>(a, p);
        default: return launch_fwd_t<16>(a, p);
    }
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
