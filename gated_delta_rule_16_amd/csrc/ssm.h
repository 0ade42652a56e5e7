// Pieces shared by the selective scan's kernels (forward, backward, token).
//
// Lane layout of the sequence kernels.  A wave is four rows of 16 lanes.  The
// 16 lanes of a row are 16 channels; a lane holds NS neighbouring states of
// its channel, and NG = 1, 2 or 4 rows share a channel (NS NG >= N: 4 states a
// lane up to N = 16, then 8 and 16), so a wave runs CW = 64 / NG channels and
// the workgroup's NG running waves WC = 64.
// Four more waves of the workgroup stage the tokens to come in LDS (Delta and
// Delta x once per channel, B and C in fp32) and finish those that are done,
// so the running waves meet no global access in their token loop.
// B_t[n] is then the same for all lanes of a row: one register holds it for
// 16 / NS tokens (lane k NS + j of row r: token k, state NS (r % NG) + j), and
// every product takes its factor by a DPP row broadcast, as part of the
// instruction, with no read of LDS.  The sum over a channel's states crosses
// rows: permlane swaps, 6 instructions for 4 tokens at NG = 4.
// States n >= N have A = B = C = 0 and stay 0.
#pragma once

#include <utility>

#include "block_launch.h"
#include "rows.h"

namespace gdr {

// Value of lane l ^ M (M = 1, 2, 4, 8): DPP moves, no LDS traffic.
template <int M>
__device__ __forceinline__ float xor_lane(float x) {
    const int i = __builtin_bit_cast(int, x);
    constexpr int ctrl = M == 1 ? 0xB1 : M == 2 ? 0x4E : 0x128;
    if constexpr (M != 4)
        return __builtin_bit_cast(float,
                                  __builtin_amdgcn_update_dpp(0, i, ctrl, 0xF, 0xF, false));
    static_assert(M == 1 || M == 2 || M == 4 || M == 8, "lane distance");
    // banks 0 and 2 of a row read 4 lanes up (row_shl 4), banks 1 and 3 down
    const int up = __builtin_amdgcn_update_dpp(0, i, 0x104, 0xF, 0x5, false);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(up, i, 0x114, 0xF, 0xA, false));
}

// One step of a halving reduction over a row of 16 lanes: lanes with bit BIT
// clear keep a's sum over the pair of lanes, lanes with it set b's.  The pair
// is l and l ^ 8, l ^ 7, l ^ 2, l ^ 1 for bits 3, 2, 1, 0: each of them one DPP
// operand, and together they reach all 16 lanes.
template <int BIT>
__device__ __forceinline__ float pair_lane(float x) {
    constexpr int ctrl = BIT == 3 ? 0x128 : BIT == 2 ? 0x141 : BIT == 1 ? 0x4E : 0xB1;
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                         0, __builtin_bit_cast(int, x), ctrl, 0xF, 0xF, false));
}
template <int BIT>
__device__ __forceinline__ float fold(float a, float b, bool bit) {
    return (bit ? b : a) + pair_lane<BIT>(bit ? a : b);
}

// The same across 16 or 32 lanes, one swap and one add.
__device__ __forceinline__ float fold16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a),
                                                    __builtin_bit_cast(unsigned, b), false, false);
    return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}
__device__ __forceinline__ float fold32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a),
                                                    __builtin_bit_cast(unsigned, b), false, false);
    return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}

// Lane I of the lane's row of 16, in every lane (a DPP operand of the
// instruction that uses it).
template <int I>
__device__ __forceinline__ float row_bcast(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                         0, __builtin_bit_cast(int, x), 0x150 + I, 0xF, 0xF, true));
}

// Fused adds with a row broadcast as their DPP operand, which the compiler does
// not form from a broadcast and an fma, 4 per block.  The wait states between
// a vector write of C and its DPP read are kept inside each block; what a block
// writes waits as long before state_sums swaps it (row_dots).
//
// h0 .. h3 += C[I .. I + 3] x0 .. x3.
template <int I>
__device__ __forceinline__ void row_fma4(float& h0, float& h1, float& h2, float& h3, float C,
                                         float x0, float x1, float x2, float x3) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %4, %5 row_newbcast:%c9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %4, %6 row_newbcast:%c10 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %4, %7 row_newbcast:%c11 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %4, %8 row_newbcast:%c12 row_mask:0xf bank_mask:0xf"
        : "+&v"(h0), "+&v"(h1), "+&v"(h2), "+&v"(h3)
        : "v"(C), "v"(x0), "v"(x1), "v"(x2), "v"(x3), "n"(I), "n"(I + 1), "n"(I + 2),
          "n"(I + 3));
}
// s (+)= C[I .. I + 3] . (x0 .. x3).
template <int I, bool FIRST>
__device__ __forceinline__ void row_dot4(float& s, float C, float x0, float x1, float x2, float x3) {
    if constexpr (FIRST)
        asm("s_nop 1\n\t"
            "v_mul_f32_dpp %0, %1, %2 row_newbcast:%c6 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%c7 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %4 row_newbcast:%c8 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%c9 row_mask:0xf bank_mask:0xf"
            : "=&v"(s)
            : "v"(C), "v"(x0), "v"(x1), "v"(x2), "v"(x3), "n"(I), "n"(I + 1), "n"(I + 2),
              "n"(I + 3));
    else
        asm("s_nop 1\n\t"
            "v_fmac_f32_dpp %0, %1, %2 row_newbcast:%c6 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%c7 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %4 row_newbcast:%c8 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%c9 row_mask:0xf bank_mask:0xf"
            : "+&v"(s)
            : "v"(C), "v"(x0), "v"(x1), "v"(x2), "v"(x3), "n"(I), "n"(I + 1), "n"(I + 2),
              "n"(I + 3));
}

// h[j] += C[j] x[j] of one token whose C starts at lane I, j from Q on.
template <int NS, int I, int Q = 0>
__device__ __forceinline__ void row_fma_each(float (&h)[NS], float C, const float (&x)[NS]) {
    row_fma4<I + Q>(h[Q], h[Q + 1], h[Q + 2], h[Q + 3], C, x[Q], x[Q + 1], x[Q + 2], x[Q + 3]);
    if constexpr (Q + 4 < NS) row_fma_each<NS, I, Q + 4>(h, C, x);
}
// h[j] += C[j] x.
template <int NS, int I, int Q = 0>
__device__ __forceinline__ void row_fma(float (&h)[NS], float C, float x) {
    row_fma4<I + Q>(h[Q], h[Q + 1], h[Q + 2], h[Q + 3], C, x, x, x, x);
    if constexpr (Q + 4 < NS) row_fma<NS, I, Q + 4>(h, C, x);
}
// sum_j C[j] h[j].
template <int NS, int I, int Q = 0>
__device__ __forceinline__ float row_dot(float C, const float (&h)[NS], float s = 0.f) {
    row_dot4<I + Q, Q == 0>(s, C, h[Q], h[Q + 1], h[Q + 2], h[Q + 3]);
    if constexpr (Q + 4 < NS) s = row_dot<NS, I, Q + 4>(C, h, s);
    return s;
}

// The four tokens of a register of C at NS = 4, in one block.
__device__ __forceinline__ void row_dot_tokens(float (&s)[4], float C, const float (&h)[4][4]) {
#define DOT4(o, a, b, c, d, i, j, k, l)                                                     \
    "v_mul_f32_dpp " o ", %4, " a " row_newbcast:" i " row_mask:0xf bank_mask:0xf\n\t"      \
    "v_fmac_f32_dpp " o ", %4, " b " row_newbcast:" j " row_mask:0xf bank_mask:0xf\n\t"     \
    "v_fmac_f32_dpp " o ", %4, " c " row_newbcast:" k " row_mask:0xf bank_mask:0xf\n\t"     \
    "v_fmac_f32_dpp " o ", %4, " d " row_newbcast:" l " row_mask:0xf bank_mask:0xf\n\t"
    asm("s_nop 1\n\t" DOT4("%0", "%5", "%6", "%7", "%8", "0", "1", "2", "3")
            DOT4("%1", "%9", "%10", "%11", "%12", "4", "5", "6", "7")
                DOT4("%2", "%13", "%14", "%15", "%16", "8", "9", "10", "11")
                    DOT4("%3", "%17", "%18", "%19", "%20", "12", "13", "14", "15") "s_nop 1"
        : "=&v"(s[0]), "=&v"(s[1]), "=&v"(s[2]), "=&v"(s[3])
        : "v"(C), "v"(h[0][0]), "v"(h[0][1]), "v"(h[0][2]), "v"(h[0][3]), "v"(h[1][0]),
          "v"(h[1][1]), "v"(h[1][2]), "v"(h[1][3]), "v"(h[2][0]), "v"(h[2][1]), "v"(h[2][2]),
          "v"(h[2][3]), "v"(h[3][0]), "v"(h[3][1]), "v"(h[3][2]), "v"(h[3][3]));
#undef DOT4
}

// Four tokens' sums over their lane's states, C in 16 / NS tokens per register.
template <int NS>
__device__ __forceinline__ void row_dots(float (&s)[4], const float (&C)[NS / 4],
                                         const float (&h)[4][NS]) {
    if constexpr (NS == 4) {
        row_dot_tokens(s, C[0], h);
    } else {
        constexpr int KT = 16 / NS;
        s[0] = row_dot<NS, NS * (0 % KT)>(C[0 / KT], h[0]);
        s[1] = row_dot<NS, NS * (1 % KT)>(C[1 / KT], h[1]);
        s[2] = row_dot<NS, NS * (2 % KT)>(C[2 / KT], h[2]);
        s[3] = row_dot<NS, NS * (3 % KT)>(C[3 / KT], h[3]);
        // what asm wrote must not be swapped at once
        asm("s_nop 1" : "+v"(s[0]), "+v"(s[1]), "+v"(s[2]), "+v"(s[3]));
    }
}

// The decays and additions of one token: K is its place in the register Bq.
template <int NS, int K, size_t... J>
__device__ __forceinline__ void scan_terms(float (&ea)[NS], float (&bx)[NS], const float (&A2)[NS],
                                           float d, float dx, float Bq,
                                           std::index_sequence<J...>) {
    ((ea[J] = __builtin_amdgcn_exp2f(d * A2[J])), ...);
    ((bx[J] = row_bcast<K * NS + J>(Bq) * dx), ...);
}

// Sums s[k] (token k of 4) over the rows of each channel and stores them at
// dst[k * pitch].  row = lane / 16.
template <int NG>
__device__ __forceinline__ void state_sums(const float (&s)[4], int row, float* dst, int pitch) {
    if constexpr (NG == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k * pitch] = s[k];
    } else {
        const float p0 = fold16(s[0], s[1]), p1 = fold16(s[2], s[3]);
        if constexpr (NG == 2) {
            dst[(row & 1) * pitch] = p0;
            dst[(2 + (row & 1)) * pitch] = p1;
        } else {
            dst[row * pitch] = fold32(p0, p1);
        }
    }
}

// Register of B or C for tokens tt .. tt + 16 / NS - 1 of a tile in LDS
// ([token][NP] floats): this lane's element.
template <int NS, int NG>
__device__ __forceinline__ float row_coef(const float* tile, int tt, int lane) {
    constexpr int NP = NS * NG;
    const int i = lane & 15;
    return tile[(tt + i / NS) * NP + NS * ((lane >> 4) % NG) + i % NS];
}

// NS states of one lane in memory ([.., N] floats, element-aligned).  Without
// RAG valid is 0 or NS.
template <int NS, bool RAG = true>
__device__ __forceinline__ void states_load(float (&h)[NS], const float* p, int valid) {
    if constexpr (RAG) {
        param_load<NS>(h, p, valid);
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = 0.f;
        if (valid > 0) param_load<NS>(h, p, NS);
    }
}
template <int NS>
__device__ __forceinline__ void states_store(float* p, const float (&h)[NS], int valid) {
    if (valid >= NS) {
#pragma unroll
        for (int i = 0; i < NS; i += 4)
            *reinterpret_cast<f32x4_e4*>(p + i) = f32x4_e4{h[i], h[i + 1], h[i + 2], h[i + 3]};
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (i < valid) p[i] = h[i];
    }
}

// The exponent's rate per unit of Delta, A log2 e.  -inf becomes fp32's lowest
// value (so A = -inf, and finite A below -2.36e38, act as -2.36e38): a step of 0,
// which padded tokens and empty sums have, then leaves the state as it is, and a
// decayed state's gradient 0 stays 0, where 0 x inf would be NaN.  NaN stays NaN.
__device__ __forceinline__ float decay_rate(float A) {
    const float r = A * kLog2e;
    return r < -3.402823466e38f ? -3.402823466e38f : r;
}

constexpr int WC = 64;   // channels per workgroup

// The first channel, in its group of Dg, of a workgroup's WC.  Where Dg is no
// multiple of 8 the last block is moved back to end with the group, so that the
// rows of all blocks are loaded and stored whole; what it then shares with the
// block before it comes out the same from both.  RAG, for groups of fewer than
// WC channels, loads element by element instead.
template <bool RAG> __device__ __forceinline__ int64_t first_channel(int64_t blk, int64_t Dg) {
    return !RAG && Dg % 8 != 0 && blk * WC > Dg - WC ? Dg - WC : blk * WC;
}

// Groups of 4 of B and C: 64 channels and the states of a token are staged by
// threads that each hold 4 states.  Where N is no multiple of 4 the last group
// starts at N - 4; with NG = 1 (N <= 4) it is loaded element by element.
template <int NG> __device__ __forceinline__ int quad_start(int64_t N, int qn) {
    return NG == 1 || 4 * qn + 4 <= N ? 4 * qn : (int)N - 4;
}
template <int NG> __device__ __forceinline__ int quad_valid(int64_t N, int qn) {
    return NG == 1 ? (int)N : 4 * qn < N ? 4 : 0;
}
// Group q = token * NP / 4 + qn of a tile [token][NP] in LDS.
template <int NP, int NG>
__device__ __forceinline__ void quad_write(float* tile, int q, int64_t N, const float (&f)[4]) {
    if (NG == 1 || N % 4 == 0) {
        *reinterpret_cast<float4*>(&tile[4 * q]) = float4{f[0], f[1], f[2], f[3]};
    } else {
        const int qn = q % (NP / 4);
        float* p = tile + q / (NP / 4) * NP + quad_start<NG>(N, qn);
        if (4 * qn < N) {
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = f[e];
        }
    }
}
// The states n >= N of ROWS rows of NP, which quad_write leaves alone where N
// is no multiple of 4.
template <int NP, int ROWS>
__device__ __forceinline__ void quad_clear(float* rows, int64_t N, int tid) {
    for (int i = tid; i < ROWS * NP; i += 256)
        if (i % NP >= N) rows[i] = 0.f;
}

// The step Delta of a token and channel, and of E channels (one branch for
// all, so their chains interleave).
__device__ __forceinline__ float ssm_delta(float raw, bool sp) { return sp ? softplus(raw) : raw; }
template <int E>
__device__ __forceinline__ void ssm_deltas(float (&d)[E], const float (&raw)[E], bool sp) {
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] = raw[e];
    if (sp) {
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] = softplus(d[e]);
    }
}

// v[e] times z[e] sigmoid(z[e]).
template <int E>
__device__ __forceinline__ void ssm_gate(float (&v)[E], const float (&z)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= z[e] * sigmoid(z[e]);
}

// Valid states of a lane that starts at state n0.
template <int NS>
__device__ __forceinline__ int states_valid(int64_t N, int n0) {
    const int64_t v = N - n0;
    return v < 0 ? 0 : v > NS ? NS : (int)v;
}

__device__ __forceinline__ int ssm_left(int64_t lim, int64_t c, int e) {
    const int64_t v = lim - c;
    return v < 0 ? 0 : v > e ? e : (int)v;
}

// h = exp2(A2 sum) h + end, over `count` segments: their end states (`ends`, at
// this lane's states) and sums of Delta, `step` floats apart.  The loads of a
// batch are in flight together: a segment costs 0.1 us, one by one 0.33.
template <int NS>
__device__ __forceinline__ void compose(float (&h)[NS], const float (&A2)[NS], const float* ends,
                                        int64_t end_step, const float* sums, int64_t sum_step,
                                        int64_t count, bool live) {
    constexpr int U = 32 / NS;
    for (int64_t s = 0; s < count; s += U) {
        // past the last: a decay of 1 and nothing added
        float e[U][NS], sd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = live && s + u < count;
            states_load<NS, false>(e[u], ends + (in ? (s + u) * end_step : 0), in);
            sd[u] = in ? sums[(s + u) * sum_step] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NS; ++j)
                h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(A2[j] * sd[u]), h[j], e[u][j]);
    }
}

}  // namespace gdr
