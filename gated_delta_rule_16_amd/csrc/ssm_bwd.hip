// gdr_ssm_scan_bwd: reverse mode of the selective scan.  With dy_t the
// gradient of the ungated output (dout_t z_t sigmoid(z_t), or dout_t), a_t =
// exp(Delta_t A) and g_t the gradient of the state,
//
//   g_t = C_t dy_t + a_{t+1} g_{t+1},            dC_t = sum_c h_t dy_t,
//   dB_t = sum_c g_t Delta_t x_t,                p_t = g_t a_t h_{t-1},
//   dx_t = Delta_t sum_n g_t B_t + D dy_t,       dA = sum_t p_t Delta_t,
//   dDelta_t = x_t sum_n g_t B_t + sum_n p_t A,  dz_t = dout_t y_t (z sigmoid(z))',
//
// Two passes.  The first runs the state forward and keeps it every S tokens
// (block_tokens; 16 at N = 16: 8 bytes of traffic per state and 16 tokens).  The
// second goes backwards over blocks of S tokens: it runs a block's states
// again from the kept one, leaving h_t and a_t of all S tokens in registers
// (128 of them), then walks the block backwards.  Lanes are laid out as in
// the forward (ssm.h).  Sums over the states cross rows with permlane swaps;
// sums over channels (dB, dC) are halving reductions over a row's 16 lanes
// (22 operations a token for the 8 values of a lane at NS = 4), then over the
// workgroup's waves in LDS, and leave as one partial per workgroup, added by
// ssm_bwd_reduce in a fixed order.  B 4 T 4096 D 2048 N 16, gated, bf16: 594 us,
// of which the first pass 159 (vector ALU busy in all cycles), the second 414
// (in 85%: the rest waits for LDS at the ends of blocks) and the sums 19.
//
// Segments: both passes run all segments of a sequence side by side.  The
// first starts every segment from zero and also forms the gradient that the
// segment alone sends to its start, sum_t (prod a) C_t dy_t, from running
// products; the second composes a segment's true start state and end
// gradient from those and adds exp(A sum Delta) h_in to each kept state.
#include <type_traits>

#include "ssm.h"

namespace gdr {

namespace {

// Tokens per block of the second pass, and between kept states: what fills
// 128 registers with h and a, and half of that where few states leave a
// workgroup few running waves, so that two fit a compute unit.
template <int NS, int NG> constexpr int block_tokens() { return NG < 4 ? 8 : 64 / NS; }

// First pass.  GAM: more than one segment.  As in the forward, NG waves run
// the states while four stage the tiles to come.
template <int NS, int NG, bool GAM, bool BF16, bool RAG>
__global__ __launch_bounds__(64 * (NG + 4)) void ssm_bwd_states_kernel(SsmBwdArgs a, int64_t nblk,
                                                                       int64_t nseg, int64_t L) {
    constexpr int NP = NS * NG, CW = WC / NG;
    constexpr int EPT = 8;
    constexpr int TT = 256 * EPT / WC;
    constexpr int TPR = WC / EPT;
    constexpr int NQ = TT * NP / 4;
    constexpr int QPT = (2 * NQ + 255) / 256;
    constexpr int KT = 16 / NS;
    constexpr int S = block_tokens<NS, NG>();
    __shared__ float2 dd[2][TT][WC];
    __shared__ __align__(16) float bc[2][2][TT * NP];
    __shared__ float ds[2][GAM ? TT : 1][WC];

    const int lane = threadIdx.x & 63, tid = (int)threadIdx.x - 64 * NG;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool scans = wv < NG;
    int64_t id = blockIdx.x;
    const int64_t blk = id % nblk;
    id /= nblk;
    const int64_t g = id % a.G;
    id /= a.G;
    const int64_t seg = id % nseg, b = id / nseg;
    const int64_t Dg = a.D / a.G, cg = g * Dg;
    const int64_t c0 = first_channel<RAG>(blk, Dg);
    const int64_t t0 = seg * L, t1 = t0 + L < a.T ? t0 + L : a.T;
    const int64_t tiles = (t1 - t0 + TT - 1) / TT;
    const int64_t nsub = (a.T + S - 1) / S;

    if (scans) {
        const int row = lane >> 4, n0 = NS * (row % NG);
        const int chl = wv * CW + (lane & 15) + 16 * (row / NG);
        const bool live = c0 + chl < Dg;
        const int64_t ch = cg + (live ? c0 + chl : 0);
        const int nv = live ? states_valid<NS>(a.N, n0) : 0;
        float A2[NS], h[NS], P[NS], gam[NS];
        param_load<NS>(A2, a.A + ch * a.N + n0, nv);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            A2[j] = decay_rate(A2[j]);
            h[j] = gam[j] = 0.f;
            P[j] = 1.f;
        }
        if (a.h0 && seg == 0) states_load<NS>(h, a.h0 + (b * a.D + ch) * a.N + n0, nv);
        float sumd = 0.f;
        __syncthreads();
        for (int64_t i = 0; i < tiles; ++i) {
            const int buf = (int)(i & 1);
            const int64_t tb = t0 + i * TT;
            const int nt = t1 - tb < TT ? (int)(t1 - tb) : TT;
            for (int tt = 0; tt < nt; tt += 4) {
                if (((tb + tt) & (S - 1)) == 0) {
                    const int64_t o = (b * nsub + (tb + tt) / S) * a.D + ch;
                    states_store<NS>(a.ckpt + o * NP + n0, h, live ? NS : 0);
                    if (GAM && live && n0 == 0) a.csum[o] = sumd;
                }
                float Bq[4 / KT], Cq[4 / KT], dy[4] = {0.f, 0.f, 0.f, 0.f};
                float2 d[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    d[k] = dd[buf][tt + k][chl];
                    if constexpr (GAM) dy[k] = ds[buf][tt + k][chl];
                }
#pragma unroll
                for (int k = 0; k < 4 / KT; ++k) {
                    Bq[k] = row_coef<NS, NG>(bc[buf][0], tt + k * KT, lane);
                    Cq[k] = GAM ? row_coef<NS, NG>(bc[buf][1], tt + k * KT, lane) : 0.f;
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
                    for (int j = 0; j < NS; ++j) h[j] = __builtin_fmaf(ea[k][j], h[j], bx[k][j]);
                }
                if constexpr (GAM) {
                    // gam += P C dy: P in place of the decays, then the
                    // products with dy, then C by broadcast
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int j = 0; j < NS; ++j) {
                            P[j] *= ea[k][j];
                            ea[k][j] = P[j] * dy[k];
                        }
                    }
                    row_fma_each<NS, NS * (0 % KT)>(gam, Cq[0 / KT], ea[0]);
                    row_fma_each<NS, NS * (1 % KT)>(gam, Cq[1 / KT], ea[1]);
                    row_fma_each<NS, NS * (2 % KT)>(gam, Cq[2 / KT], ea[2]);
                    row_fma_each<NS, NS * (3 % KT)>(gam, Cq[3 / KT], ea[3]);
                    sumd += (d[0].x + d[1].x) + (d[2].x + d[3].x);
                }
            }
            __syncthreads();
        }
        if constexpr (GAM) {
            const int64_t o = (b * nseg + seg) * a.D + ch;
            states_store<NS>(a.hend + o * NP + n0, h, live ? NS : 0);
            states_store<NS>(a.gstart + o * NP + n0, gam, live ? NS : 0);
            if (live && n0 == 0) a.sdelta[o] = sumd;
        }
        return;
    }

    const int srow = tid / TPR, sc = (tid % TPR) * EPT;
    const int sv = ssm_left(Dg, c0 + sc, EPT);
    const int64_t scg = cg + c0 + sc;
    float bias[EPT];
    param_load<EPT>(bias, a.bias + scg, a.bias ? sv : 0);
    // addresses of the next tile to fetch
    using T = typename std::conditional<BF16, bf16_t, float>::type;
    const T* px = static_cast<const T*>(a.x) + b * a.xb + (t0 + srow) * a.xt + scg;
    const T* pt = static_cast<const T*>(a.dt) + b * a.dtb + (t0 + srow) * a.dtt + scg;
    const T* pz = static_cast<const T*>(a.z) + b * a.zb + (t0 + srow) * a.zt + scg;
    int64_t po = b * a.ob + (t0 + srow) * a.ot + scg;
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
        Row<EPT, true, RAG> o16;
        Row<EPT, false, RAG> o32;
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
        if constexpr (GAM) {
            r.o16.load(a.dout, po, a.dout_bf16 ? v : 0);
            r.o32.load(a.dout, po, a.dout_bf16 ? 0 : v);
            r.z.load(pz, 0, a.z ? v : 0);
            po += TT * a.ot;
            pz += TT * a.zt;
        }
#pragma unroll
        for (int j = 0; j < QPT; ++j) {
            const int q = tid + 256 * j;
            const bool isc = q >= NQ;
            if (isc && !GAM) continue;
            const int qt = (q % NQ) / (NP / 4), qn = q % (NP / 4);
            const int vq = q < 2 * NQ && qt < left ? quad_valid<NG>(a.N, qn) : 0;
            r.q[j].load(pq[j], 0, vq);
            pq[j] += TT * (isc ? a.ct : a.bt);
        }
    };
    auto stage = [&](int64_t i, const Rows& rows) {
        const int buf = (int)(i & 1);
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
        if constexpr (GAM) {
            float o[EPT], z[EPT];
            if (a.dout_bf16)
                rows.o16.unpack(o);
            else
                rows.o32.unpack(o);
            rows.z.unpack(z);
            if (a.z) ssm_gate(o, z);
#pragma unroll
            for (int e = 0; e < EPT; ++e) ds[buf][srow][sc + e] = o[e];
        }
#pragma unroll
        for (int q4 = 0; q4 < QPT; ++q4) {
            const int q = tid + 256 * q4;
            if (q >= 2 * NQ || (q >= NQ && !GAM)) continue;
            float f[4];
            rows.q[q4].unpack(f);
            quad_write<NP, NG>(bc[buf][q >= NQ], q % NQ, a.N, f);
        }
    };
    quad_clear<NP, 4 * TT>(&bc[0][0][0], a.N, tid);
    fetch(0, rows0);
    fetch(1, rows1);
    stage(0, rows0);
    fetch(2, rows0);
    __syncthreads();
    auto step = [&](int64_t i, Rows& rows) {
        if (i + 1 < tiles) {
            stage(i + 1, rows);
            fetch(i + 3, rows);
        }
        __syncthreads();
    };
    for (int64_t i = 0; i < tiles; i += 2) {
        step(i, rows1);
        if (i + 1 < tiles) step(i + 1, rows0);
    }
}

// A token of the second pass, backwards: gr enters as a_{t+1} g_{t+1} and
// leaves as a_t g_t; I is the token's place in Bq and Cq.
template <int NS, int I>
__device__ __forceinline__ void back_token(float (&gr)[NS], float (&dA)[NS], float (&pv)[2 * NS],
                                           float& sB, float& sA, const float (&aa)[NS],
                                           const float (&hh)[NS], const float (&hp)[NS],
                                           const float (&A2)[NS], float d, float dx, float dy,
                                           float Bq, float Cq, bool own) {
    row_fma<NS, I>(gr, Cq, dy);
    const float ody = own ? dy : 0.f, odx = own ? dx : 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        pv[j] = hh[j] * ody;
        pv[NS + j] = gr[j] * odx;
    }
    sB = row_dot<NS, I>(Bq, gr);
    sA = 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        gr[j] *= aa[j];
        const float u = gr[j] * hp[j];
        sA = j == 0 ? u * A2[j] : __builtin_fmaf(u, A2[j], sA);
        dA[j] = __builtin_fmaf(u, d, dA[j]);
    }
}

// The first two steps of a halving reduction over a row of 16 lanes, 8 values
// to 2: lane bits 3 and 2 tell banks of 4 lanes apart, so a DPP add under a
// bank mask writes each half, two instructions a value and no select.  Lanes
// are left with values (v[0], v[1]) + 4 (lane bit 3) + 2 (lane bit 2).  Every
// operand of a DPP read is written three instructions or more before it.
__device__ __forceinline__ void row_fold_8(float (&q)[2], const float (&v)[8]) {
    float t0, t1, t2, t3;
#define BOTH(o, x, y, pair, lo, hi)                                                      \
    "v_add_f32_dpp " o ", " x ", " x " " pair " row_mask:0xf bank_mask:" lo "\n\t"       \
    "v_add_f32_dpp " o ", " y ", " y " " pair " row_mask:0xf bank_mask:" hi "\n\t"
    asm("s_nop 1\n\t" BOTH("%2", "%6", "%10", "row_ror:8", "0x3", "0xc")
            BOTH("%4", "%8", "%12", "row_ror:8", "0x3", "0xc")
                BOTH("%3", "%7", "%11", "row_ror:8", "0x3", "0xc")
                    BOTH("%5", "%9", "%13", "row_ror:8", "0x3", "0xc")
                        BOTH("%0", "%2", "%4", "row_half_mirror", "0x5", "0xa")
                            BOTH("%1", "%3", "%5", "row_half_mirror", "0x5", "0xa") "s_nop 1"
        : "=&v"(q[0]), "=&v"(q[1]), "=&v"(t0), "=&v"(t1), "=&v"(t2), "=&v"(t3)
        : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]),
          "v"(v[7]));
#undef BOTH
}

// Sums of a token pair's values (the token at q, and the next) over a wave's
// channels: pv[0 .. NS) for dC, the rest for dB.  Lane bits 3 .. 0 choose what
// a lane is left with; at NS = 4 bit 0 chooses the token.  Lanes (and rows, NG
// < 4) that are left with the same sum store it twice.
template <int NS, int NG>
__device__ __forceinline__ void channel_sums(float (*p)[2 * NS * NG], const float (&p0)[2 * NS],
                                             const float (&p1)[2 * NS], int lane, int n0) {
    constexpr int NP = NS * NG;
    const int half = ((lane >> 3) & 1) * NP + n0;
    auto rows = [](float x) {
        if constexpr (NG <= 2) x = fold32(x, x);
        if constexpr (NG <= 1) x = fold16(x, x);
        return x;
    };
    if constexpr (NS == 4) {
        float q0[2], q1[2];
        row_fold_8(q0, p0);
        row_fold_8(q1, p1);
        const float a = fold<1>(q0[0], q0[1], lane & 2), b = fold<1>(q1[0], q1[1], lane & 2);
        p[lane & 1][half + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1)] =
            rows(fold<0>(a, b, lane & 1));
    } else {
        // 8 values at a time: of dC and dB the states 4 i .. 4 i + 3, folded to 2
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float(&pv)[2 * NS] = k ? p1 : p0;
            float w[NS / 4];
#pragma unroll
            for (int i = 0; i < NS / 4; ++i) {
                const float v[8] = {pv[4 * i],          pv[4 * i + 1],      pv[4 * i + 2],
                                    pv[4 * i + 3],      pv[NS + 4 * i],     pv[NS + 4 * i + 1],
                                    pv[NS + 4 * i + 2], pv[NS + 4 * i + 3]};
                float q[2];
                row_fold_8(q, v);
                w[i] = fold<1>(q[0], q[1], lane & 2);
            }
            // bit 0 chooses the group of four states of a pair of groups
#pragma unroll
            for (int i = 0; i < NS / 8; ++i)
                p[k][half + 8 * i + 4 * (lane & 1) + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1)] =
                    rows(fold<0>(w[2 * i], w[2 * i + 1], lane & 1));
        }
    }
}

// Second pass.  NG waves run the blocks, backwards; the other four stage the
// next block meanwhile and finish the last one: its gradients from the sums
// over n, which the running waves leave in the block's place in st.
template <int NS, int NG, bool BF16, bool RAG>
__global__ __launch_bounds__(64 * (NG + 4), NS == 16 ? 1 : 2) void ssm_bwd_kernel(SsmBwdArgs a,
                                                                                  int64_t nblk,
                                                                                  int64_t nseg,
                                                                                  int64_t L) {
    constexpr int NP = NS * NG, CW = WC / NG;
    constexpr int S = block_tokens<NS, NG>();
    constexpr int EPT = S * WC / 256;
    constexpr int TPR = WC / EPT;
    constexpr int NQ = S * NP / 4;
    constexpr int QPT = (2 * NQ + 255) / 256;
    constexpr int KT = 16 / NS;
    constexpr int WP = WC + 16;               // pitch: 4 tokens' sums meet no bank twice
    // Delta, Delta x, dy and a place for y; the sums over n of g B and of p A
    // take the place of Delta and Delta x
    __shared__ __align__(16) float st[2][4][S][WP];
    __shared__ __align__(16) float bc[2][2][S * NP];
    __shared__ float pbc[2][NG][S][2 * NP];   // each wave's sums over its channels: dC, dB

    const int lane = threadIdx.x & 63, tid = (int)threadIdx.x - 64 * NG;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool runs = wv < NG;
    int64_t id = blockIdx.x;
    const int64_t blk = id % nblk;
    id /= nblk;
    const int64_t g = id % a.G;
    id /= a.G;
    const int64_t seg = id % nseg, b = id / nseg;
    const int64_t Dg = a.D / a.G, cg = g * Dg;
    const int64_t c0 = first_channel<RAG>(blk, Dg);
    const int64_t t0 = seg * L, t1 = t0 + L < a.T ? t0 + L : a.T;
    const int64_t nsub = (a.T + S - 1) / S;
    const int64_t first = t0 / S, last = (t1 + S - 1) / S - 1;
    float* const part = a.part + (b * nseg + seg) * a.D * (a.N + 2);

    if (runs) {
        const int row = lane >> 4, n0 = NS * (row % NG);
        const int chl = wv * CW + (lane & 15) + 16 * (row / NG);
        const bool live = c0 + chl < Dg;
        // a channel that the block shares with the one before counts there
        const bool own = c0 + chl >= blk * WC;
        const int64_t ch = cg + (live ? c0 + chl : 0);
        const int nv = live ? states_valid<NS>(a.N, n0) : 0;
        float A2[NS], hin[NS], gr[NS], dA[NS];
        param_load<NS>(A2, a.A + ch * a.N + n0, nv);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            A2[j] = decay_rate(A2[j]);
            hin[j] = gr[j] = dA[j] = 0.f;
        }
        const int64_t so = (b * a.D + ch) * a.N + n0;
        // the segment's start state (segment 0's kept states hold h0 already)
        if (seg > 0) {
            const int64_t o = b * nseg * a.D + ch;
            states_load<NS, false>(hin, a.hend + o * NP + n0, live);
            compose<NS>(hin, A2, a.hend + (o + a.D) * NP + n0, a.D * NP, a.sdelta + o + a.D, a.D,
                        seg - 1, live);
        }
        // gr = a_{t+1} g_{t+1} past the segment's last token
        if (a.dh_final) states_load<NS>(gr, a.dh_final + so, nv);
        if (seg < nseg - 1) {
            const int64_t o = (b * nseg + nseg - 1) * a.D + ch;
            compose<NS>(gr, A2, a.gstart + o * NP + n0, -a.D * NP, a.sdelta + o, -a.D,
                        nseg - 1 - seg, live);
        }
        float kept[NS], ksum = 0.f;
        auto fetch = [&](int64_t sub) {
            const int64_t ko = (b * nsub + sub) * a.D + ch;
            states_load<NS, false>(kept, a.ckpt + ko * NP + n0, live);
            if (seg > 0) ksum = live ? a.csum[ko] : 0.f;
        };
        fetch(last);
        __syncthreads();
        for (int64_t sub = last; sub >= first; --sub) {
            const int buf = (int)(sub & 1);
            float hs[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j)
                hs[j] = seg > 0
                            ? __builtin_fmaf(__builtin_amdgcn_exp2f(A2[j] * ksum), hin[j], kept[j])
                            : kept[j];
            // operands of 4 tokens, read before the group in front of them
            // writes its sums, so that their latency is covered
            struct Operands {
                float d[4], dx[4], dy[4], Bq[4 / KT], Cq[4 / KT];
            };
            auto read = [&](Operands& o, int tt, bool back) {
#pragma unroll
                for (int k = 0; k < 4 / KT; ++k) {
                    o.Bq[k] = row_coef<NS, NG>(bc[buf][0], tt + k * KT, lane);
                    o.Cq[k] = row_coef<NS, NG>(bc[buf][1], tt + k * KT, lane);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o.d[k] = st[buf][0][tt + k][chl];
                    o.dx[k] = st[buf][1][tt + k][chl];
                    if (back) o.dy[k] = st[buf][2][tt + k][chl];
                }
            };
            // the block's states again, all kept in registers
            constexpr auto js = std::make_index_sequence<NS>{};
            float hh[S][NS], aa[S][NS];
            Operands o;
            read(o, 0, S == 4);
#pragma unroll
            for (int tt = 0; tt < S; tt += 4) {
                Operands next;
                if (tt + 4 < S) read(next, tt + 4, tt + 8 >= S);
#define TOKEN(k) \
    scan_terms<NS, k % KT>(aa[tt + k], hh[tt + k], A2, o.d[k], o.dx[k], o.Bq[k / KT], js)
                TOKEN(0);
                TOKEN(1);
                TOKEN(2);
                TOKEN(3);
#undef TOKEN
#pragma unroll
                for (int k = tt; k < tt + 4; ++k) {
#pragma unroll
                    for (int j = 0; j < NS; ++j)
                        hh[k][j] =
                            __builtin_fmaf(aa[k][j], k ? hh[k ? k - 1 : 0][j] : hs[j], hh[k][j]);
                }
                if (a.z) {
                    float s[4], h4[4][NS];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int j = 0; j < NS; ++j) h4[k][j] = hh[tt + k][j];
                    row_dots<NS>(s, o.Cq, h4);
                    state_sums<NG>(s, row, &st[buf][3][tt][chl], WP);
                }
                if (tt + 4 < S) o = next;
            }
            // and backwards, from the last group, whose operands are here
#pragma unroll
            for (int tt = S - 4; tt >= 0; tt -= 4) {
                // half of the kept states are done with: the next block's
                // start takes their registers (short blocks load it at once)
                if (tt == (S == 16 ? 4 : S - 4) && sub > first) fetch(sub - 1);
                Operands next;
                if (tt > 0) read(next, tt - 4, true);
                float sB[4], sA[4], pv[4][2 * NS];
#define TOKEN(k)                                                                               \
    back_token<NS, NS*(k % KT)>(gr, dA, pv[k], sB[k], sA[k], aa[tt + k], hh[tt + k],           \
                                tt + k == 0 ? hs : hh[tt + k == 0 ? 0 : tt + k - 1], A2,       \
                                o.d[k], o.dx[k], o.dy[k], o.Bq[k / KT], o.Cq[k / KT], own)
                TOKEN(3);
                TOKEN(2);
                channel_sums<NS, NG>(&pbc[buf][wv][tt + 2], pv[2], pv[3], lane, n0);
                TOKEN(1);
                TOKEN(0);
                channel_sums<NS, NG>(&pbc[buf][wv][tt], pv[0], pv[1], lane, n0);
#undef TOKEN
                asm("s_nop 1" : "+v"(sB[0]), "+v"(sB[1]), "+v"(sB[2]), "+v"(sB[3]));
                state_sums<NG>(sB, row, &st[buf][0][tt][chl], WP);
                state_sums<NG>(sA, row, &st[buf][1][tt][chl], WP);
                if (tt > 0) o = next;
            }
            __syncthreads();
        }
        if (seg == 0 && a.dh0) states_store<NS>(a.dh0 + so, gr, nv);
        states_store<NS>(part + ch * a.N + n0, dA, nv);
        __syncthreads();
        return;
    }

    const int srow = tid / TPR, sc = (tid % TPR) * EPT;
    const int sv = ssm_left(Dg, c0 + sc, EPT);
    const int64_t scg = cg + c0 + sc;
    float dD[EPT], dbias[EPT], bias[EPT], skip[EPT];
    small_load<EPT>(bias, a.bias + scg, a.bias ? sv : 0);
    small_load<EPT>(skip, a.D_skip + scg, a.D_skip ? sv : 0);
#pragma unroll
    for (int e = 0; e < EPT; ++e) dD[e] = dbias[e] = 0.f;

    // addresses of the next block to fetch
    using T = typename std::conditional<BF16, bf16_t, float>::type;
    const T* px = static_cast<const T*>(a.x) + b * a.xb + (last * S + srow) * a.xt + scg;
    const T* pt = static_cast<const T*>(a.dt) + b * a.dtb + (last * S + srow) * a.dtt + scg;
    const T* pz = static_cast<const T*>(a.z) + b * a.zb + (last * S + srow) * a.zt + scg;
    int64_t po = b * a.ob + (last * S + srow) * a.ot + scg;
    const T* pq[QPT];
#pragma unroll
    for (int i = 0; i < QPT; ++i) {
        const int q = tid + 256 * i, qt = (q % NQ) / (NP / 4), qn = q % (NP / 4);
        pq[i] = q >= NQ ? static_cast<const T*>(a.Cm) + b * a.cb + (last * S + qt) * a.ct
                        : static_cast<const T*>(a.Bm) + b * a.bb + (last * S + qt) * a.bt;
        pq[i] += g * a.N + quad_start<NG>(a.N, qn);
    }
    // two blocks' loads are in flight, each in its own registers
    struct Rows {
        Row<EPT, BF16, RAG> x, t, z;
        Row<EPT, true, RAG> o16;
        Row<EPT, false, RAG> o32;
        Row<4, BF16, NG == 1> q[QPT];
    } rows0, rows1;
    auto fetch = [&](int64_t sub, Rows& r) {
        if (sub < first) return;
        const int left = t1 - sub * S < S ? (int)(t1 - sub * S) : S;
        const int v = srow < left ? sv : 0;
        r.x.load(px, 0, v);
        r.t.load(pt, 0, v);
        r.o16.load(a.dout, po, a.dout_bf16 ? v : 0);
        r.o32.load(a.dout, po, a.dout_bf16 ? 0 : v);
        r.z.load(pz, 0, a.z ? v : 0);
        px -= S * a.xt;
        pt -= S * a.dtt;
        po -= S * a.ot;
        pz -= S * a.zt;
#pragma unroll
        for (int j = 0; j < QPT; ++j) {
            const int q = tid + 256 * j;
            const bool isc = q >= NQ;
            const int qt = (q % NQ) / (NP / 4), qn = q % (NP / 4);
            const int vq = q < 2 * NQ && qt < left ? quad_valid<NG>(a.N, qn) : 0;
            r.q[j].load(pq[j], 0, vq);
            pq[j] -= S * (isc ? a.ct : a.bt);
        }
    };
    // of a staged block, until it is finished: x, Delta, its derivative, dy, and
    // dout (z sigmoid(z))'
    struct Held {
        float x[EPT], d[EPT], ddr[EPT], dy[EPT], og[EPT];
    };
    auto stage = [&](int64_t sub, const Rows& rows, Held& k) {
        const int buf = (int)(sub & 1);
        const int v = sub * S + srow < t1 ? sv : 0;
        float r[EPT], z[EPT];
        rows.x.unpack(k.x);
        rows.t.unpack(r);
        if (a.dout_bf16)
            rows.o16.unpack(k.dy);
        else
            rows.o32.unpack(k.dy);
        rows.z.unpack(z);
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            r[e] += bias[e];
            k.ddr[e] = 1.f;
        }
        if (a.softplus) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) softplus_grad(r[e], k.d[e], k.ddr[e]);
        } else {
#pragma unroll
            for (int e = 0; e < EPT; ++e) k.d[e] = r[e];
        }
        if (a.z) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                const float sg = sigmoid(z[e]);
                k.og[e] = k.dy[e] * sg * __builtin_fmaf(z[e], 1.f - sg, 1.f);
                k.dy[e] *= z[e] * sg;
            }
        }
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            k.d[e] = (RAG ? e < v : v > 0) ? k.d[e] : 0.f;
            st[buf][0][srow][sc + e] = k.d[e];
            st[buf][1][srow][sc + e] = k.d[e] * k.x[e];
            st[buf][2][srow][sc + e] = k.dy[e];
        }
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int q = tid + 256 * i;
            if (q >= 2 * NQ) continue;
            float f[4];
            rows.q[i].unpack(f);
            quad_write<NP, NG>(bc[buf][q >= NQ], q % NQ, a.N, f);
        }
    };
    int64_t oo = (b * a.T + last * S + srow) * a.D + scg;
    constexpr int PPT = (S * 2 * NP + 255) / 256;     // sums of dC and dB per thread
    const int64_t bct = a.G * 2 * NP;                 // and the partials of a token
    float* pbo = a.bcpart + ((blk * a.B + b) * a.T + last * S) * bct + g * 2 * NP;
    auto finish = [&](int64_t sub, const Held& k) {
        const int buf = (int)(sub & 1);
        const int left = t1 - sub * S < S ? (int)(t1 - sub * S) : S;
        const int v = srow < left ? sv : 0;
        if (v > 0) {
            float dxv[EPT], dtv[EPT], dzv[EPT];
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                const float gB = st[buf][0][srow][sc + e], pA = st[buf][1][srow][sc + e];
                dxv[e] = __builtin_fmaf(k.d[e], gB, skip[e] * k.dy[e]);
                // a padded token's sums with a rate of fp32's lowest value may overflow
                dtv[e] = k.ddr[e] == 0.f
                             ? 0.f
                             : __builtin_fmaf(k.x[e], gB, pA * kLn2) * k.ddr[e];
                if (a.z)
                    dzv[e] = k.og[e] * __builtin_fmaf(skip[e], k.x[e], st[buf][3][srow][sc + e]);
                if (!RAG || e < v) {
                    dD[e] = __builtin_fmaf(k.dy[e], k.x[e], dD[e]);
                    dbias[e] += dtv[e];
                }
            }
            row_store<EPT, RAG>(a.dx, oo, a.grad_bf16, dxv, v);
            row_store<EPT, RAG>(a.ddt, oo, a.grad_bf16, dtv, v);
            if (a.z) row_store<EPT, RAG>(a.dz, oo, a.grad_bf16, dzv, v);
        }
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
            const int q = (tid + 256 * i) / (2 * NP), c = (tid + 256 * i) % (2 * NP);
            if (q >= left) continue;
            float s = pbc[buf][0][q][c];
#pragma unroll
            for (int w = 1; w < NG; ++w) s += pbc[buf][w][q][c];
            pbo[q * bct + c] = s;
        }
        oo -= S * a.D;
        pbo -= S * bct;
    };
    Held even, odd;
    quad_clear<NP, 4 * S>(&bc[0][0][0], a.N, tid);
    fetch(last, rows0);
    fetch(last - 1, rows1);
    stage(last, rows0, even);
    fetch(last - 2, rows0);
    __syncthreads();
    // while block sub runs, block sub - 1 is staged (in the buffers of block
    // sub + 1, finished already) and block sub - 3's loads are issued
    auto step = [&](int64_t sub, const Held& now, Held& next, Rows& rows) {
        if (sub > first) {
            stage(sub - 1, rows, next);
            fetch(sub - 3, rows);
        }
        __syncthreads();
        finish(sub, now);
    };
    for (int64_t sub = last; sub >= first; sub -= 2) {
        step(sub, even, odd, rows1);
        if (sub > first) step(sub - 1, odd, even, rows0);
    }
    // dD and dbias over the thread rows of a channel, through the buffer that
    // the last block did not use (block `first` may not be finished yet)
    float* red = &st[(first & 1) ^ 1][0][0][0];
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

// dB, dC [B, T, G, N] = the sum of the channel blocks' partials (the first
// nbc workgroups), and dA, dD, ddt_bias = the sum of the P = B nseg partial rows
// of D (N + 2) columns (the others: 64 columns each, four waves taking every
// fourth row).  Fixed orders; one launch, since both are short.
template <int NP>
__global__ __launch_bounds__(256) void ssm_bwd_reduce(SsmBwdArgs a, int64_t nblk, int64_t nbc,
                                                      int64_t P) {
    __shared__ float red[4][64];
    if (blockIdx.x < nbc) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = a.B * a.T * a.G * 2 * NP;
        if (i >= n) return;
        const int j = (int)(i % NP);
        const int64_t row = i / (2 * NP);
        if (j >= a.N) return;
        float s = 0.f;
        for (int64_t k = 0; k < nblk; ++k) s += a.bcpart[k * n + i];
        float f[1] = {s};
        row_store<1>((i / NP) & 1 ? a.dB : a.dC, row * a.N + j, a.grad_bf16, f, 1);
        return;
    }
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t M = a.D * (a.N + 2), m = ((int64_t)blockIdx.x - nbc) * 64 + lane;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (m < M) {
        for (int64_t p = wv; p < P; p += 16)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (p + 4 * u < P) s[u] += a.part[(p + 4 * u) * M + m];
    }
    red[wv][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (wv == 0 && m < M) {
        const float v = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
        const int64_t d = m - a.D * a.N;
        if (d < 0) a.dA[m] = v;
        else if (d < a.D) { if (a.dD) a.dD[d] = v; }
        else if (a.dbias) a.dbias[d - a.D] = v;
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Segments of the backward: up to two workgroups per compute unit (B 4 T 4096
// D 2048 N 16: 587 us with 512 workgroups, 630 with 256, 780 with 384).
SsmPlan bwd_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    SsmPlan p;
    p.nblk = cdiv(D / G, 64);
    int64_t n = 512 / (B * G * p.nblk);
    const int64_t most = ssm_most_segments(T);
    if (n > most) n = most;
    if (n < 1) n = 1;
    p.L = cdiv(cdiv(T, n), 32) * 32;
    p.nseg = T > 0 ? cdiv(T, p.L) : 1;
    return p;
}

// Tokens between kept states, for N states (block_tokens).
int64_t kept_tokens(int64_t N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 8 : 4; }

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
    const int64_t nsub = cdiv(T, kept_tokens(N));
    const bool many = p.nseg > 1;
    const int64_t NP = ssm_padded_states(N);
    l.ckpt = take(B * nsub * D * NP);
    l.csum = take(many ? B * nsub * D : 0);
    l.hend = take(many ? B * p.nseg * D * NP : 0);
    l.gstart = take(many ? B * p.nseg * D * NP : 0);
    l.sdelta = take(many ? B * p.nseg * D : 0);
    l.part = take(B * p.nseg * D * (N + 2));
    l.bcpart = take(p.nblk * B * T * G * 2 * NP);
    l.total = at;
    return l;
}

template <int NS, int NG, bool BF16, bool RAG>
hipError_t launch_bwd_r(const SsmBwdArgs& a, const SsmPlan& p) {
    const dim3 grid((unsigned)(a.B * a.G * p.nblk * p.nseg)), threads(64 * (NG + 4));
    if (p.nseg > 1)
        hipLaunchKernelGGL((ssm_bwd_states_kernel<NS, NG, true, BF16, RAG>), grid, threads, 0,
                           a.stream, a, p.nblk, p.nseg, p.L);
    else
        hipLaunchKernelGGL((ssm_bwd_states_kernel<NS, NG, false, BF16, RAG>), grid, threads, 0,
                           a.stream, a, p.nblk, p.nseg, p.L);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ssm_bwd_kernel<NS, NG, BF16, RAG>), grid, threads, 0, a.stream, a, p.nblk,
                       p.nseg, p.L);
    return hipGetLastError();
}

template <int NS, int NG>
hipError_t launch_bwd_t(const SsmBwdArgs& a, const SsmPlan& p) {
    const int64_t Dg = a.D / a.G;
    const bool rag = Dg % 8 != 0 && Dg < WC;
    hipError_t e;
    if (a.in_bf16)
        e = rag ? launch_bwd_r<NS, NG, true, true>(a, p) : launch_bwd_r<NS, NG, true, false>(a, p);
    else
        e = rag ? launch_bwd_r<NS, NG, false, true>(a, p)
                : launch_bwd_r<NS, NG, false, false>(a, p);
    if (e != hipSuccess) return e;
    const int64_t nbc = cdiv(a.B * a.T * a.G * 2 * NS * NG, 256);
    hipLaunchKernelGGL((ssm_bwd_reduce<NS * NG>), dim3((unsigned)(nbc + cdiv(a.D * (a.N + 2), 64))),
                       dim3(256), 0, a.stream, a, p.nblk, nbc, a.B * p.nseg);
    return hipGetLastError();
}

}  // namespace

size_t ssm_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    return bwd_layout(bwd_plan(B, T, D, G, N), B, T, D, G, N).total;
}

int64_t ssm_bwd_workgroups(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    const SsmPlan p = bwd_plan(B, T, D, G, N);
    const int64_t n = 2 * B * G * p.nblk * p.nseg;    // of 512 threads
    const int64_t r = cdiv(B * T * G * 2 * ssm_padded_states(N), 256) + cdiv(D * (N + 2), 64);
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
    if (a.N <= 4) return launch_bwd_t<4, 1>(a, p);
    if (a.N <= 8) return launch_bwd_t<4, 2>(a, p);
    if (a.N <= 16) return launch_bwd_t<4, 4>(a, p);
    if (a.N <= 32) return launch_bwd_t<8, 4>(a, p);
    return launch_bwd_t<16, 4>(a, p);
}

}  // namespace gdr
