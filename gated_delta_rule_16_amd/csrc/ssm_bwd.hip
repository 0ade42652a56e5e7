// gdr_ssm_scan_bwd: reverse mode of the selective scan.  With dy_t the
// gradient of the ungated output (dout_t z_t sigmoid(z_t), or dout_t), a_t =
// exp(Delta_t A) and g_t the gradient of the state,
//
//   g_t = C_t dy_t + a_{t+1} g_{t+1},            dC_t = sum_c h_t dy_t,
//   dB_t = sum_c g_t Delta_t x_t,                p_t = g_t a_t h_{t-1},
//   dx_t = Delta_t sum_n g_t B_t + D dy_t,       dA = sum_t p_t Delta_t,
//   dDelta_t = x_t sum_n g_t B_t + sum_n p_t A,  dz_t = dout_t y_t (z sigmoid(z))',
//
// Two passes.  The first runs the state forward and keeps it every S = 16
// tokens (8 bytes per state and 16 tokens of traffic instead of a state per
// token).  The second goes backwards over blocks of S tokens: it runs a
// block's states again from the kept one, leaving h_t and a_t of all S tokens
// in registers (128 of them), then walks the block backwards.  Sums over the
// states are halving reductions over a channel's lanes, 4 tokens together;
// sums over channels (dB, dC) are halving reductions over the wave (8 values,
// 16 lane operations at N = 16), then over the workgroup's waves in LDS, and
// leave as one partial per workgroup, added by ssm_bc_reduce in a fixed order.
//
// Segments: both passes run all segments of a sequence side by side.  The
// first starts every segment from zero and also forms the gradient that the
// segment alone sends to its start, sum_t (prod a) C_t dy_t, from running
// products; the second composes a segment's true start state and end
// gradient from those and adds exp(A sum Delta) h_in to each kept state.
#include "ssm.h"

namespace gdr {

namespace {

// Tokens per block of the second pass.
template <int LPC> constexpr int block_tokens() { return LPC == 1 ? 8 : 16; }

// First pass.  GAM: more than one segment.
template <int LPC, bool GAM>
__global__ __launch_bounds__(256) void ssm_bwd_states_kernel(SsmBwdArgs a, int64_t nblk,
                                                             int64_t nseg, int64_t L) {
    constexpr int WC = 256 / LPC;
    constexpr int TT = 8 * LPC < 32 ? 8 * LPC : 32;
    constexpr int EPT = TT * WC / 256;
    constexpr int TPR = WC / EPT;
    constexpr int NQ = TT * LPC;
    constexpr int QPT = (2 * NQ + 255) / 256;
    constexpr int S = block_tokens<LPC>();
    __shared__ float2 dd[TT][WC];
    __shared__ float4 bc[TT][2][LPC];
    __shared__ float ds[GAM ? TT : 1][WC];

    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    int64_t id = blockIdx.x;
    const int64_t blk = id % nblk;
    id /= nblk;
    const int64_t g = id % a.G;
    id /= a.G;
    const int64_t seg = id % nseg, b = id / nseg;
    const int64_t Dg = a.D / a.G, c0 = blk * WC, cg = g * Dg;
    const int64_t t0 = seg * L, t1 = t0 + L < a.T ? t0 + L : a.T;
    const int64_t nsub = (a.T + S - 1) / S;

    const int ng = lane % LPC, chl = wv * (64 / LPC) + lane / LPC;
    const bool live = c0 + chl < Dg;
    const int64_t ch = cg + (live ? c0 + chl : 0);
    const int nv = live ? ssm_states(a.N, ng) : 0;
    float A2[4], h[4] = {0.f, 0.f, 0.f, 0.f}, P[4] = {1.f, 1.f, 1.f, 1.f};
    float gam[4] = {0.f, 0.f, 0.f, 0.f};
    param_load<4>(A2, a.A + ch * a.N + 4 * ng, nv);
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[j] *= kLog2e;
    if (a.h0 && seg == 0) state_load(h, a.h0 + (b * a.D + ch) * a.N + 4 * ng, nv);

    const int srow = tid / TPR, sc = (tid % TPR) * EPT;
    const int sv = ssm_left(Dg, c0 + sc, EPT);
    const int64_t scg = cg + c0 + sc;
    float bias[EPT];
#pragma unroll
    for (int e = 0; e < EPT; ++e) bias[e] = a.bias && e < sv ? a.bias[scg + e] : 0.f;
    RawRow<EPT> rx, rt, rz, ro;
    RawRow<4> rq[QPT];
    auto fetch = [&](int64_t tb) {
        const int64_t t = tb + srow;
        const int v = t < t1 ? sv : 0;
        row_load<EPT>(rx, a.x, v ? b * a.xb + t * a.xt + scg : 0, a.in_bf16, v);
        row_load<EPT>(rt, a.dt, v ? b * a.dtb + t * a.dtt + scg : 0, a.in_bf16, v);
        if constexpr (GAM) {
            row_load<EPT>(ro, a.dout, v ? b * a.ob + t * a.ot + scg : 0, a.dout_bf16, v);
            if (a.z) row_load<EPT>(rz, a.z, v ? b * a.zb + t * a.zt + scg : 0, a.in_bf16, v);
        }
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int q = tid + 256 * i;
            const bool isc = q >= NQ;
            if (isc && !GAM) continue;
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
        const bool tok = tb + srow < t1;
        float x[EPT], r[EPT];
        row_unpack<EPT>(x, rx, a.in_bf16);
        row_unpack<EPT>(r, rt, a.in_bf16);
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            float d = ssm_delta(r[e] + bias[e], a.softplus);
            d = tok && e < sv ? d : 0.f;
            dd[srow][sc + e] = float2{d, d * x[e]};
        }
        if constexpr (GAM) {
            float o[EPT], z[EPT];
            row_unpack<EPT>(o, ro, a.dout_bf16);
            if (a.z) row_unpack<EPT>(z, rz, a.in_bf16);
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                if (a.z) o[e] *= z[e] * sigmoid(z[e]);
                ds[srow][sc + e] = o[e];
            }
        }
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int q = tid + 256 * i;
            const bool isc = q >= NQ;
            if (q >= 2 * NQ || (isc && !GAM)) continue;
            float f[4];
            row_unpack<4>(f, rq[i], a.in_bf16);
            bc[(q % NQ) / LPC][isc][q % LPC] = float4{f[0], f[1], f[2], f[3]};
        }
        __syncthreads();
        if (tb + TT < t1) fetch(tb + TT);
        const int nt = t1 - tb < TT ? (int)(t1 - tb) : TT;
        for (int tt = 0; tt < nt; tt += 4) {
            if (((tb + tt) & (S - 1)) == 0) {
                const int64_t o = (b * nsub + (tb + tt) / S) * a.D + ch;
                state_store(a.ckpt + o * a.N + 4 * ng, h, nv);
                if (GAM && live && ng == 0) a.csum[o] = sumd;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 d = dd[tt + k][chl];
                const float4 B4 = bc[tt + k][0][ng];
                const float Bv[4] = {B4.x, B4.y, B4.z, B4.w};
                float aa[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    aa[j] = __builtin_amdgcn_exp2f(d.x * A2[j]);
                    h[j] = __builtin_fmaf(aa[j], h[j], d.y * Bv[j]);
                }
                if constexpr (GAM) {
                    const float dy = ds[tt + k][chl];
                    const float4 C4 = bc[tt + k][1][ng];
                    const float Cv[4] = {C4.x, C4.y, C4.z, C4.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        P[j] *= aa[j];
                        gam[j] = __builtin_fmaf(P[j], Cv[j] * dy, gam[j]);
                    }
                    sumd += d.x;
                }
            }
        }
        __syncthreads();
    }
    if constexpr (GAM) {
        const int64_t o = (b * nseg + seg) * a.D + ch;
        state_store(a.hend + o * a.N + 4 * ng, h, nv);
        state_store(a.gstart + o * a.N + 4 * ng, gam, nv);
        if (live && ng == 0) a.sdelta[o] = sumd;
    }
}

// Halving reduction over the channels of a wave: v holds 8 values per lane
// (index i) and token; afterwards each lane holds the sum over its wave's
// channels of value `idx` (returned by sum_index) in v[0] (and v[1] at LPC 16).
template <int LPC>
__device__ __forceinline__ void wave_channel_sums(float (&v)[8], int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fold32(v[i], v[i + 4]);
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = fold16(v[i], v[i + 2]);
    if constexpr (LPC <= 8) v[0] = fold<8>(v[0], v[1], lane & 8);
    if constexpr (LPC <= 4) v[0] += xor_lane<4>(v[0]);
    if constexpr (LPC <= 2) v[0] += xor_lane<2>(v[0]);
    if constexpr (LPC <= 1) v[0] += xor_lane<1>(v[0]);
}

// Second pass.
template <int LPC>
__global__ __launch_bounds__(256) void ssm_bwd_kernel(SsmBwdArgs a, int64_t nblk, int64_t nseg,
                                                      int64_t L) {
    constexpr int WC = 256 / LPC;
    constexpr int S = block_tokens<LPC>();
    constexpr int EPT = S * WC / 256;
    constexpr int TPR = WC / EPT;
    constexpr int NQ = S * LPC;
    constexpr int QPT = (2 * NQ + 255) / 256;
    constexpr int NP = 4 * LPC;
    __shared__ float4 st[S][WC];              // Delta, Delta x, dy, (y); then sums over n
    __shared__ float4 bc[S][2][LPC];
    __shared__ float pbc[4][S][2 * NP];       // each wave's sums over its channels: dC, dB

    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    int64_t id = blockIdx.x;
    const int64_t blk = id % nblk;
    id /= nblk;
    const int64_t g = id % a.G;
    id /= a.G;
    const int64_t seg = id % nseg, b = id / nseg;
    const int64_t Dg = a.D / a.G, c0 = blk * WC, cg = g * Dg;
    const int64_t t0 = seg * L, t1 = t0 + L < a.T ? t0 + L : a.T;
    const int64_t nsub = (a.T + S - 1) / S;

    const int ng = lane % LPC, chl = wv * (64 / LPC) + lane / LPC;
    const bool live = c0 + chl < Dg;
    const int64_t ch = cg + (live ? c0 + chl : 0);
    const int nv = live ? ssm_states(a.N, ng) : 0;
    float A2[4], hin[4] = {0.f, 0.f, 0.f, 0.f}, gr[4] = {0.f, 0.f, 0.f, 0.f};
    float dA[4] = {0.f, 0.f, 0.f, 0.f};
    param_load<4>(A2, a.A + ch * a.N + 4 * ng, nv);
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[j] *= kLog2e;
    const int64_t so = (b * a.D + ch) * a.N + 4 * ng;
    // the segment's start state (segment 0's kept states hold h0 already)
    for (int64_t s = 0; s < seg; ++s) {
        const int64_t o = (b * nseg + s) * a.D + ch;
        float e[4];
        state_load(e, a.hend + o * a.N + 4 * ng, nv);
        const float sd = live ? a.sdelta[o] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            hin[j] = s == 0 ? e[j] : __builtin_fmaf(__builtin_amdgcn_exp2f(A2[j] * sd), hin[j], e[j]);
    }
    // gr = a_{t+1} g_{t+1} past the segment's last token
    if (a.dh_final) state_load(gr, a.dh_final + so, nv);
    for (int64_t s = nseg - 1; s > seg; --s) {
        const int64_t o = (b * nseg + s) * a.D + ch;
        float e[4];
        state_load(e, a.gstart + o * a.N + 4 * ng, nv);
        const float sd = live ? a.sdelta[o] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            gr[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(A2[j] * sd), gr[j], e[j]);
    }

    const int srow = tid / TPR, sc = (tid % TPR) * EPT;
    const int sv = ssm_left(Dg, c0 + sc, EPT);
    const int64_t scg = cg + c0 + sc;
    float bias[EPT], skip[EPT], dD[EPT], dbias[EPT];
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
        bias[e] = a.bias && e < sv ? a.bias[scg + e] : 0.f;
        skip[e] = a.D_skip && e < sv ? a.D_skip[scg + e] : 0.f;
        dD[e] = dbias[e] = 0.f;
    }

    const int64_t first = t0 / S, last = (t1 + S - 1) / S;
    for (int64_t sub = last - 1; sub >= first; --sub) {
        const int64_t tb = sub * S, t = tb + srow;
        const int v = t < t1 ? sv : 0;
        RawRow<EPT> rx, rt, rz, ro;
        RawRow<4> rq[QPT];
        row_load<EPT>(rx, a.x, v ? b * a.xb + t * a.xt + scg : 0, a.in_bf16, v);
        row_load<EPT>(rt, a.dt, v ? b * a.dtb + t * a.dtt + scg : 0, a.in_bf16, v);
        row_load<EPT>(ro, a.dout, v ? b * a.ob + t * a.ot + scg : 0, a.dout_bf16, v);
        if (a.z) row_load<EPT>(rz, a.z, v ? b * a.zb + t * a.zt + scg : 0, a.in_bf16, v);
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int q = tid + 256 * i;
            const bool isc = q >= NQ;
            const int qt = (q % NQ) / LPC, qn = q % LPC;
            const int64_t tq = tb + qt;
            const int vq = q < 2 * NQ && tq < t1 ? ssm_states(a.N, qn) : 0;
            row_load<4>(rq[i], isc ? a.Cm : a.Bm,
                        vq ? (isc ? b * a.cb + tq * a.ct : b * a.bb + tq * a.bt) + g * a.N + 4 * qn
                           : 0,
                        a.in_bf16, vq);
        }
        const int64_t ko = (b * nsub + sub) * a.D + ch;
        float hs[4];
        state_load(hs, a.ckpt + ko * a.N + 4 * ng, nv);
        if (seg > 0) {
            const float sd = live ? a.csum[ko] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                hs[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(A2[j] * sd), hin[j], hs[j]);
        }
        {
            float x[EPT], r[EPT], o[EPT], z[EPT];
            row_unpack<EPT>(x, rx, a.in_bf16);
            row_unpack<EPT>(r, rt, a.in_bf16);
            row_unpack<EPT>(o, ro, a.dout_bf16);
            if (a.z) row_unpack<EPT>(z, rz, a.in_bf16);
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                float d = ssm_delta(r[e] + bias[e], a.softplus);
                d = e < v ? d : 0.f;
                if (a.z) o[e] *= z[e] * sigmoid(z[e]);
                st[srow][sc + e] = float4{d, d * x[e], o[e], 0.f};
            }
        }
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int q = tid + 256 * i;
            if (q >= 2 * NQ) continue;
            float f[4];
            row_unpack<4>(f, rq[i], a.in_bf16);
            bc[(q % NQ) / LPC][q >= NQ][q % LPC] = float4{f[0], f[1], f[2], f[3]};
        }
        __syncthreads();

        // the block's states again, all kept in registers
        float hh[S][4], aa[S][4];
#pragma unroll
        for (int tt = 0; tt < S; tt += 4) {
            float s[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 d = st[tt + k][chl];
                const float4 B4 = bc[tt + k][0][ng], C4 = bc[tt + k][1][ng];
                const float Bv[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = tt + k == 0 ? hs[j] : hh[tt + k == 0 ? 0 : tt + k - 1][j];
                    aa[tt + k][j] = __builtin_amdgcn_exp2f(d.x * A2[j]);
                    hh[tt + k][j] = __builtin_fmaf(aa[tt + k][j], p, d.y * Bv[j]);
                }
                s[k] = __builtin_fmaf(C4.w, hh[tt + k][3], __builtin_fmaf(C4.z, hh[tt + k][2],
                       __builtin_fmaf(C4.y, hh[tt + k][1], C4.x * hh[tt + k][0])));
            }
            if (a.z) channel_sums<LPC>(s, ng, &st[tt][chl].w, 4 * WC);
        }
        // and backwards
        float dAl[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int tt = S - 4; tt >= 0; tt -= 4) {
            float sB[4], sA[4];
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const int q = tt + k;
                const float4 d = st[q][chl];
                const float4 B4 = bc[q][0][ng], C4 = bc[q][1][ng];
                const float Bv[4] = {B4.x, B4.y, B4.z, B4.w};
                const float Cv[4] = {C4.x, C4.y, C4.z, C4.w};
                float pv[8];
                sB[k] = sA[k] = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = q == 0 ? hs[j] : hh[q == 0 ? 0 : q - 1][j];
                    gr[j] = __builtin_fmaf(Cv[j], d.z, gr[j]);
                    pv[j] = hh[q][j] * d.z;
                    pv[4 + j] = gr[j] * d.y;
                    sB[k] = __builtin_fmaf(gr[j], Bv[j], sB[k]);
                    gr[j] *= aa[q][j];
                    const float u = gr[j] * p;
                    sA[k] = __builtin_fmaf(u, A2[j], sA[k]);
                    dAl[j] = __builtin_fmaf(u, d.x, dAl[j]);
                }
                wave_channel_sums<LPC>(pv, lane);
                // lane bits 5, 4 (and 3) chose the value: C or B, then its index
                if constexpr (LPC == 16) {
                    const int i0 = ((lane >> 5) & 1) * NP + 4 * ng + ((lane >> 4) & 1) * 2;
                    pbc[wv][q][i0] = pv[0];
                    pbc[wv][q][i0 + 1] = pv[1];
                } else {
                    const int i0 = ((lane >> 5) & 1) * NP + 4 * ng + ((lane >> 4) & 1) * 2 +
                                   ((lane >> 3) & 1);
                    if ((lane & 7) < LPC) pbc[wv][q][i0] = pv[0];
                }
            }
            channel_sums<LPC>(sB, ng, &st[tt][chl].x, 4 * WC);
            channel_sums<LPC>(sA, ng, &st[tt][chl].y, 4 * WC);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) dA[j] += dAl[j];
        __syncthreads();

        if (v > 0) {
            float x[EPT], r[EPT], o[EPT], z[EPT], dxv[EPT], dtv[EPT];
            row_unpack<EPT>(x, rx, a.in_bf16);
            row_unpack<EPT>(r, rt, a.in_bf16);
            row_unpack<EPT>(o, ro, a.dout_bf16);
            if (a.z) row_unpack<EPT>(z, rz, a.in_bf16);
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                const float4 q = st[srow][sc + e];
                const float raw = r[e] + bias[e];
                const float d = ssm_delta(raw, a.softplus);
                float dy = o[e];
                if (a.z) {
                    const float sg = sigmoid(z[e]);
                    const float y = __builtin_fmaf(skip[e], x[e], q.w);
                    dy *= z[e] * sg;
                    z[e] = o[e] * y * sg * __builtin_fmaf(z[e], 1.f - sg, 1.f);
                }
                dxv[e] = __builtin_fmaf(d, q.x, skip[e] * dy);
                float dr = __builtin_fmaf(x[e], q.x, q.y * kLn2);
                if (a.softplus) dr *= sigmoid(raw);
                dtv[e] = dr;
                if (e < v) {
                    dD[e] = __builtin_fmaf(dy, x[e], dD[e]);
                    dbias[e] += dr;
                }
            }
            const int64_t oo = (b * a.T + t) * a.D + scg;
            row_store<EPT>(a.dx, oo, a.grad_bf16, dxv, v);
            row_store<EPT>(a.ddt, oo, a.grad_bf16, dtv, v);
            if (a.z) row_store<EPT>(a.dz, oo, a.grad_bf16, z, v);
        }
        for (int i = tid; i < S * 2 * NP; i += 256) {
            const int q = i / (2 * NP), k = i % (2 * NP);
            if (tb + q < t1)
                a.bcpart[(((blk * a.B + b) * a.T + tb + q) * a.G + g) * 2 * NP + k] =
                    (pbc[0][q][k] + pbc[1][q][k]) + (pbc[2][q][k] + pbc[3][q][k]);
        }
        __syncthreads();
    }
    if (seg == 0 && a.dh0) state_store(a.dh0 + so, gr, nv);
    float* part = a.part + (b * nseg + seg) * a.D * (a.N + 2);
    state_store(part + ch * a.N + 4 * ng, dA, nv);
    // dD and dbias over the thread rows of a channel, through st
    float* red = reinterpret_cast<float*>(st);
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
        red[srow * 2 * WC + sc + e] = dD[e];
        red[srow * 2 * WC + WC + sc + e] = dbias[e];
    }
    __syncthreads();
    for (int i = tid; i < 2 * WC; i += 256) {
        const int c = i % WC;
        if (c0 + c >= Dg) continue;
        float s = 0.f;
        for (int q = 0; q < S; ++q) s += red[q * 2 * WC + i];
        part[a.D * a.N + (i / WC) * a.D + cg + c0 + c] = s;
    }
}

// dB, dC [B, T, G, N] = the sum of the channel blocks' partials.
template <int NP>
__global__ __launch_bounds__(256) void ssm_bc_reduce(SsmBwdArgs a, int64_t nblk) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = a.B * a.T * a.G * 2 * NP;
    if (i >= n) return;
    float s = 0.f;
    for (int64_t k = 0; k < nblk; ++k) s += a.bcpart[k * n + i];
    const int j = (int)(i % NP);
    const int64_t row = i / (2 * NP);
    if (j >= a.N) return;
    float f[1] = {s};
    row_store<1>((i / NP) & 1 ? a.dB : a.dC, row * a.N + j, a.grad_bf16, f, 1);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Segments of the backward.  Its second pass holds two waves per SIMD, so one
// segment does where the channels give 2048 waves; fewer channels get enough
// segments (of at least 64 tokens) for that.
SsmPlan bwd_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    SsmPlan p;
    p.lpc = ssm_lanes(N);
    p.nblk = cdiv(D / G, 256 / p.lpc);
    const int64_t waves = 4 * B * G * p.nblk;
    int64_t n = cdiv(2048, waves);
    const int64_t most = cdiv(T, 64);
    if (n > most) n = most;
    if (n < 1) n = 1;
    p.L = cdiv(cdiv(T, n), 32) * 32;
    p.nseg = T > 0 ? cdiv(T, p.L) : 1;
    return p;
}

struct BwdLayout {
    size_t ckpt, csum, hend, gstart, sdelta, part, bcpart, total;
};

BwdLayout bwd_layout(const SsmPlan& p, int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    BwdLayout l;
    size_t at = 0;
    auto take = [&](int64_t n) {
        const size_t o = at;
        at += (sizeof(float) * (size_t)n + 255) & ~(size_t)255;
        return o;
    };
    const int64_t nsub = cdiv(T, p.lpc == 1 ? 8 : 16);
    const bool many = p.nseg > 1;
    l.ckpt = take(B * nsub * D * N);
    l.csum = take(many ? B * nsub * D : 0);
    l.hend = take(many ? B * p.nseg * D * N : 0);
    l.gstart = take(many ? B * p.nseg * D * N : 0);
    l.sdelta = take(many ? B * p.nseg * D : 0);
    l.part = take(B * p.nseg * D * (N + 2));
    l.bcpart = take(p.nblk * B * T * G * 8 * p.lpc);
    l.total = at;
    return l;
}

template <int LPC>
hipError_t launch_bwd_t(const SsmBwdArgs& a, const SsmPlan& p) {
    const dim3 grid((unsigned)(a.B * a.G * p.nblk * p.nseg));
    if (p.nseg > 1)
        hipLaunchKernelGGL((ssm_bwd_states_kernel<LPC, true>), grid, dim3(256), 0, a.stream, a,
                           p.nblk, p.nseg, p.L);
    else
        hipLaunchKernelGGL((ssm_bwd_states_kernel<LPC, false>), grid, dim3(256), 0, a.stream, a,
                           p.nblk, p.nseg, p.L);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ssm_bwd_kernel<LPC>), grid, dim3(256), 0, a.stream, a, p.nblk, p.nseg,
                       p.L);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = a.B * a.T * a.G * 8 * LPC;
    hipLaunchKernelGGL((ssm_bc_reduce<4 * LPC>), dim3((unsigned)cdiv(n, 256)), dim3(256), 0,
                       a.stream, a, p.nblk);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_sum_partials(a.part, a.B * p.nseg, a.D * (a.N + 2), a.dA, a.D * a.N, a.dD, a.D,
                               a.dbias, a.stream);
}

}  // namespace

size_t ssm_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    return bwd_layout(bwd_plan(B, T, D, G, N), B, T, D, G, N).total;
}

int64_t ssm_bwd_workgroups(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    const SsmPlan p = bwd_plan(B, T, D, G, N);
    const int64_t n = B * G * p.nblk * p.nseg, r = cdiv(B * T * G * 8 * p.lpc, 256);
    return n > r ? n : r;
}

hipError_t launch_ssm_bwd(SsmBwdArgs a, void* ws) {
    const SsmPlan p = bwd_plan(a.B, a.T, a.D, a.G, a.N);
    const BwdLayout l = bwd_layout(p, a.B, a.T, a.D, a.G, a.N);
    char* w = static_cast<char*>(ws);
    a.ckpt = reinterpret_cast<float*>(w + l.ckpt);
    a.csum = reinterpret_cast<float*>(w + l.csum);
    a.hend = reinterpret_cast<float*>(w + l.hend);
    a.gstart = reinterpret_cast<float*>(w + l.gstart);
    a.sdelta = reinterpret_cast<float*>(w + l.sdelta);
    a.part = reinterpret_cast<float*>(w + l.part);
    a.bcpart = reinterpret_cast<float*>(w + l.bcpart);
    switch (p.lpc) {
        case 1: return launch_bwd_t<1>(a, p);
        case 2: return launch_bwd_t<2>(a, p);
        case 4: return launch_bwd_t<4>(a, p);
        case 8: return launch_bwd_t<8>(a, p);
        default: return launch_bwd_t<16>(a, p);
    }
}

}  // namespace gdr
