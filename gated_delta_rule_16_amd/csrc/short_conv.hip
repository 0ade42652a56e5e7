// gdr_short_conv_*: the short causal depthwise convolution of the block's q,
// k and v paths (and of a state space layer's input), with an optional SiLU:
//
//   u_t[c] = bias[c] + sum_{j<K} w[c][j] x_{t-K+1+j}[c],  y = u or u sigmoid(u),
//
// K = 2, 3 or 4; x before the sequence is the state (its last K - 1 inputs).
// Reverse mode, with du = dy, or dy sigmoid(u)(1 + u (1 - sigmoid(u))):
//
//   dx_i = sum_j w[j] du_{i+K-1-j},  dw[j] = sum_t x_{t-K+1+j} du_t,  dbias = sum_t du_t.
//
// All of it is bound by HBM: a channel costs 2 (3 backward) accesses against
// ~2K + 4 (6K + 8) operations.  A lane owns E neighbouring channels and walks
// along the tokens of its stretch with the last K - 1 inputs in registers, so
// every input is read once but for the K - 1 rows where stretches meet.  B 8
// T 4096 K 4 with SiLU in bf16: forward at C 6144 162 us (5.0 TB/s), backward at
// C 2048 93 us (4.3 TB/s); a copy reaches 4.9 to 5.4 on the same card.
#include "block_launch.h"
#include "rows.h"

namespace gdr {

namespace {

constexpr int E = 8;              // channels per lane: one 16-byte access in bf16
constexpr int FWD_TOKENS = 4;     // loads in flight per lane

__device__ __forceinline__ int clampi(int64_t v, int hi) {
    return v < 0 ? 0 : v > hi ? hi : (int)v;
}

// A lane's group of channels at c: how many it has.  Without RAG the last
// group of the row is moved back to end with it, and is full too.
template <int EE, bool RAG>
__device__ __forceinline__ int own_group(int64_t& c, int64_t C) {
    if constexpr (RAG) return clampi(C - c, EE);
    if (c >= C) return 0;
    if (c > C - EE) c = C - EE;
    return EE;
}

// How the lanes of a wave lie over channels and tokens.
//   WIDE: 64 groups of channels of one stretch of tokens; the token's address is
//     the wave's, in scalar registers.
//   PACKED: rows of at most 32 groups of channels: gl lanes (a power of two) to a
//     stretch, and 64 / gl stretches to a wave (bf16, K 2, B 59 T 12693 C 78:
//     47 us against 135 WIDE; at C 2048 the lanes' own token addresses would
//     cost the backward 123 us instead of 94).
//   RAGGED: the same with any number of channels, element by element at a row's
//     end: fewer channels than one group, or a state written in place.
enum Form { WIDE, PACKED, RAGGED };

// Lanes per stretch for C channels in groups of EE.
template <int EE> int group_lanes(int64_t C) {
    int gl = 1;
    while (gl < 64 && (int64_t)gl * EE < C) gl *= 2;
    return gl;
}

// Row t of [state; x] for one lane's channels: t >= 0 from x, else the state
// (or zeros without one).
template <int EE, bool BF16, bool RAG>
__device__ __forceinline__ void load_in(Row<EE, BF16, RAG>& r, const ConvArgs& a, int64_t b,
                                        int64_t t, int64_t c, int valid) {
    const bool past = t < 0;
    r.load(past ? a.s0 : a.x,
           past ? (b * (a.K - 1) + t + a.K - 1) * a.C + c : b * a.xb + t * a.xt + c,
           past && !a.s0 ? 0 : valid);
}

template <int K, bool BF16, Form FORM>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, int64_t ncb, int64_t nunit,
                                                       int TL, int gl) {
    constexpr bool RAG = FORM == RAGGED;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t id = blockIdx.x;
    const int64_t cb = id % ncb;
    id /= ncb;
    const int64_t b = id / nunit;
    int64_t st = (id % nunit) * 4 + wv, c = (cb * 64 + lane) * E;
    if constexpr (FORM != WIDE) {
        st = st * (64 / gl) + lane / gl;
        c = (cb * gl + lane % gl) * E;
    }
    const int valid = own_group<E, RAG>(c, a.C);
    const int64_t t0 = st * TL;
    if (valid == 0 || t0 >= a.T) return;
    const int64_t t1 = t0 + TL < a.T ? t0 + TL : a.T;
    float w[E * K], bias[E];
    param_load<E * K>(w, a.w + c * K, valid * K);
    param_load<E>(bias, a.bias + c, a.bias ? valid : 0);
    float win[K - 1][E];
    {
        Row<E, BF16, RAG> r[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) load_in(r[j], a, b, t0 - (K - 1) + j, c, valid);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) r[j].unpack(win[j]);
        if (t0 == 0 && a.s_final) {
            // the lane that reads the state also writes the next one, so the
            // two may be the same buffer: all K - 1 rows are read (the state
            // rows above, or x) before the first is written
            Row<E, BF16, RAG> f[K - 1];
#pragma unroll
            for (int m = 0; m < K - 1; ++m) load_in(f[m], a, b, a.T - (K - 1) + m, c, valid);
#pragma unroll
            for (int m = 0; m < K - 1; ++m)
                f[m].copy_to(a.s_final, (b * (K - 1) + m) * a.C + c, valid);
        }
    }
    for (int64_t t = t0; t < t1; t += FWD_TOKENS) {
        Row<E, BF16, RAG> r[FWD_TOKENS];
#pragma unroll
        for (int u = 0; u < FWD_TOKENS; ++u)
            r[u].load(a.x, b * a.xb + (t + u < t1 ? t + u : t1 - 1) * a.xt + c, valid);
#pragma unroll
        for (int u = 0; u < FWD_TOKENS; ++u) {
            float x[E], y[E];
            r[u].unpack(x);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float s = bias[e];
#pragma unroll
                for (int j = 0; j < K - 1; ++j) s = __builtin_fmaf(w[e * K + j], win[j][e], s);
                s = __builtin_fmaf(w[e * K + K - 1], x[e], s);
                y[e] = a.silu ? s * sigmoid(s) : s;
#pragma unroll
                for (int j = 0; j + 1 < K - 1; ++j) win[j][e] = win[j + 1][e];
                win[K - 2][e] = x[e];
            }
            if (t + u < t1)
                row_store<E, RAG>(a.y, (b * a.T + t + u) * a.C + c, a.out_bf16, y, valid);
        }
    }
}

// One decode token: the lane shifts its own channels' state.
template <int K, bool BF16>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, int64_t ncg) {
    constexpr int SE = 4;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t b = id / ncg, c = (id % ncg) * SE;
    if (b >= a.B) return;
    const int valid = clampi(a.C - c, SE);
    Row<SE, BF16, true> r[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j].load(a.s0, (b * (K - 1) + j) * a.C + c, valid);
    r[K - 1].load(a.x, b * a.xb + c, valid);
    float y[SE], x[K][SE], w[SE * K];
    param_load<SE * K>(w, a.w + c * K, valid * K);
    param_load<SE>(y, a.bias + c, a.bias ? valid : 0);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        r[j].unpack(x[j]);
#pragma unroll
        for (int e = 0; e < SE; ++e)
            y[e] = __builtin_fmaf(w[e * K + j], x[j][e], y[e]);
    }
#pragma unroll
    for (int e = 0; e < SE; ++e) y[e] = a.silu ? y[e] * sigmoid(y[e]) : y[e];
    row_store<SE>(a.y, b * a.C + c, a.out_bf16, y, valid);
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        r[j + 1].copy_to(a.s_final, (b * (K - 1) + j) * a.C + c, valid);
}

constexpr int BE = 4;             // backward: channels per lane

// Backward.  Wave wv of a workgroup walks stretch 4 i + wv; dw and dbias stay
// in registers over all of a workgroup's stretches, are joined over its waves
// through LDS and go out as one partial row [C (K + 1)] per workgroup row.
// The walk runs K - 1 tokens past the stretch to complete its last dx, and a
// stretch leaves the dx of the K - 1 rows before it to its neighbour -- but
// the first, whose earlier rows are the state's gradient.
template <int K, bool BF16, bool DY16, Form FORM>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, int64_t ncb, int64_t nrow,
                                                       int64_t nunit, int TL, int gl) {
    constexpr bool RAG = FORM == RAGGED;
    __shared__ float red[3][64][BE * (K + 1) + 1];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t cb = blockIdx.x % ncb, row = blockIdx.x / ncb;
    int64_t c = FORM == WIDE ? (cb * 64 + lane) * BE : (cb * gl + lane % gl) * BE;
    const int valid = own_group<BE, RAG>(c, a.C);
    float w[BE * K], bias[BE], dw[BE][K], db[BE];
    param_load<BE * K>(w, a.w + c * K, valid * K);
    param_load<BE>(bias, a.bias + c, a.bias ? valid : 0);
#pragma unroll
    for (int e = 0; e < BE; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[e][j] = 0.f;
    }
    const int64_t units = a.B * nunit;
    if (valid > 0)
        for (int64_t un = row; un < units; un += nrow) {
            const int64_t b = un / nunit;
            int64_t t0 = ((un % nunit) * 4 + wv) * TL;
            if constexpr (FORM != WIDE) t0 = t0 * (64 / gl) + lane / gl * TL;
            if (t0 >= a.T) continue;
            const int64_t t1 = t0 + TL < a.T ? t0 + TL : a.T;
            // x window: rows t - K + 1 .. t; du window: du_{t-K+1} .. du_t
            float win[K][BE], du[K][BE];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                Row<BE, BF16, RAG> r;
                load_in(r, a, b, t0 - (K - 1) + j, c, valid);
                r.unpack(win[j + 1]);
            }
#pragma unroll
            for (int j = 0; j < K; ++j)
#pragma unroll
                for (int e = 0; e < BE; ++e) du[j][e] = 0.f;
            const int64_t tend = t1 + K - 1;
            constexpr int U = 4;
            for (int64_t tb = t0; tb < tend; tb += U) {
                Row<BE, BF16, RAG> rx[U];
                Row<BE, DY16, RAG> rd[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t t = tb + u;
                    const int v = t < a.T && t < tend ? valid : 0;
                    rx[u].load(a.x, b * a.xb + t * a.xt + c, v);
                    rd[u].load(a.dy, b * a.yb + t * a.yt + c, v);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t t = tb + u;
                    float x[BE], d[BE];
                    rx[u].unpack(x);
                    rd[u].unpack(d);
                    const bool mine = t < t1;     // du_t counts for dw here
                    float out[BE];
#pragma unroll
                    for (int e = 0; e < BE; ++e) {
#pragma unroll
                        for (int j = 0; j + 1 < K; ++j) {
                            win[j][e] = win[j + 1][e];
                            du[j][e] = du[j + 1][e];
                        }
                        win[K - 1][e] = x[e];
                        float g = d[e];
                        if (a.silu) {
                            float s = bias[e];
#pragma unroll
                            for (int j = 0; j < K; ++j)
                                s = __builtin_fmaf(w[e * K + j], win[j][e], s);
                            const float sg = sigmoid(s);
                            g *= sg * __builtin_fmaf(s, 1.f - sg, 1.f);
                        }
                        // rows past the sequence loaded zeros, but an infinite
                        // bias would still make their g NaN
                        g = t < a.T ? g : 0.f;
                        du[K - 1][e] = g;
                        if (mine) {
                            db[e] += g;
#pragma unroll
                            for (int j = 0; j < K; ++j)
                                dw[e][j] = __builtin_fmaf(win[j][e], g, dw[e][j]);
                        }
                        // dx_{t-K+1} = sum_j w[j] du_{t-j}
                        float o = 0.f;
#pragma unroll
                        for (int j = 0; j < K; ++j)
                            o = __builtin_fmaf(w[e * K + j], du[K - 1 - j][e], o);
                        out[e] = o;
                    }
                    const int64_t i = t - (K - 1);
                    if (t >= tend || (i < t0 && t0 > 0)) continue;
                    if (a.ds_final && i >= a.T - (K - 1)) {
                        const float* p = a.ds_final +
                                         (b * (K - 1) + i - (a.T - (K - 1))) * a.C + c;
#pragma unroll
                        for (int e = 0; e < BE; ++e)
                            if (e < valid) out[e] += p[e];
                    }
                    if (i >= 0)
                        row_store<BE, RAG>(a.dx, (b * a.T + i) * a.C + c, a.grad_bf16, out, valid);
                    else if (a.ds0)
                        row_store<BE, RAG>(a.ds0, (b * (K - 1) + i + K - 1) * a.C + c, false, out,
                                      valid);
                }
            }
        }
    if (!a.part) return;
    if constexpr (FORM != WIDE) {
        // over the wave's stretches, to all of their lanes
        for (int d = gl; d < 64; d *= 2)
#pragma unroll
            for (int e = 0; e < BE; ++e) {
                db[e] += __shfl_xor(db[e], d, 64);
#pragma unroll
                for (int j = 0; j < K; ++j) dw[e][j] += __shfl_xor(dw[e][j], d, 64);
            }
    }
    if (wv > 0) {
#pragma unroll
        for (int e = 0; e < BE; ++e) {
#pragma unroll
            for (int j = 0; j < K; ++j) red[wv - 1][lane][e * K + j] = dw[e][j];
            red[wv - 1][lane][BE * K + e] = db[e];
        }
    }
    __syncthreads();
    if (wv == 0 && valid > 0 && (FORM == WIDE || lane < gl)) {
        float* p = a.part + row * a.C * (K + 1);
#pragma unroll
        for (int e = 0; e < BE; ++e) {
            if (e >= valid) break;
#pragma unroll
            for (int j = 0; j < K; ++j)
                p[(c + e) * K + j] = (dw[e][j] + red[0][lane][e * K + j]) +
                                     (red[1][lane][e * K + j] + red[2][lane][e * K + j]);
            p[a.C * K + c + e] = (db[e] + red[0][lane][BE * K + e]) +
                                 (red[1][lane][BE * K + e] + red[2][lane][BE * K + e]);
        }
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Shape {
    int64_t ncb, nunit;     // blocks of channels; of 4 waves' stretches
    int TL, gl;
};

// The launch for groups of EE channels.  A stretch of TL tokens, between lo and
// hi: long enough that the K - 1 rows read twice are few, short enough that the
// launch fills the chip: halved while it has fewer than 8192 waves.  bf16 K 4,
// forward / backward in us with 8192, 2048 and 32768: B 8 T 4096 C 6144 163 / 260,
// 172 / 260, 155 / 263; B 8 T 4096 C 2048 52 / 90, 47 / 90, 56 / 114; B 4 T 1024
// C 6144 24 / 48, 20 / 37, 24 / 48: no one bound is best for all of them.
template <int EE>
Shape shape(int64_t B, int64_t T, int64_t C, int lo, int hi) {
    Shape s;
    s.gl = group_lanes<EE>(C);
    s.ncb = cdiv(C, 64 * EE);
    const int64_t per = 64 / s.gl;              // stretches per wave
    s.TL = hi;
    while (s.TL > lo && B * s.ncb * cdiv(T, s.TL * per) < 8192) s.TL /= 2;
    s.nunit = cdiv(T, 4 * per * s.TL);
    return s;
}
Shape fwd_shape(int64_t B, int64_t T, int64_t C) { return shape<E>(B, T, C, 4, 64); }
Shape bwd_shape(int64_t B, int64_t T, int64_t C) { return shape<BE>(B, T, C, 8, 64); }

// Backward: workgroup rows (partials of dw) for the launch.
int64_t bwd_rows(const Shape& s, int64_t B) {
    const int64_t units = B * s.nunit, cap = cdiv(4096, s.ncb);
    return units < cap ? units : cap;
}

template <int K>
void fwd_t(const ConvArgs& a, dim3 grid, const Shape& s) {
    // a moved group reads channels that another lane also writes back: not where
    // the state's buffer is the next one's
    const bool rag = a.C < E || (a.C % E != 0 && a.s_final && a.s_final == a.s0);
    const bool packed = s.gl < 64;
#define FWD(BF16, FORM)                                                                           \
    hipLaunchKernelGGL((conv_fwd_kernel<K, BF16, FORM>), grid, dim3(256), 0, a.stream, a, s.ncb, \
                       s.nunit, s.TL, s.gl)
    if (a.in_bf16) {
        if (rag) FWD(true, RAGGED);
        else if (packed) FWD(true, PACKED);
        else FWD(true, WIDE);
    } else {
        if (rag) FWD(false, RAGGED);
        else if (packed) FWD(false, PACKED);
        else FWD(false, WIDE);
    }
#undef FWD
}

template <int K>
void step_t(const ConvArgs& a, dim3 grid, int64_t ncg) {
    if (a.in_bf16)
        hipLaunchKernelGGL((conv_step_kernel<K, true>), grid, dim3(256), 0, a.stream, a, ncg);
    else
        hipLaunchKernelGGL((conv_step_kernel<K, false>), grid, dim3(256), 0, a.stream, a, ncg);
}

template <int K, bool BF16, bool DY16>
void bwd_t(const ConvArgs& a, dim3 grid, const Shape& s, int64_t nrow) {
#define BWD(FORM)                                                                                \
    hipLaunchKernelGGL((conv_bwd_kernel<K, BF16, DY16, FORM>), grid, dim3(256), 0, a.stream, a, \
                       s.ncb, nrow, s.nunit, s.TL, s.gl)
    if (a.C < BE) BWD(RAGGED);
    else if (s.gl < 64) BWD(PACKED);
    else BWD(WIDE);
#undef BWD
}

template <int K>
void bwd_k(const ConvArgs& a, dim3 grid, const Shape& s, int64_t nrow) {
    if (a.in_bf16) {
        if (a.dy_bf16) bwd_t<K, true, true>(a, grid, s, nrow);
        else bwd_t<K, true, false>(a, grid, s, nrow);
    } else {
        if (a.dy_bf16) bwd_t<K, false, true>(a, grid, s, nrow);
        else bwd_t<K, false, false>(a, grid, s, nrow);
    }
}

}  // namespace

size_t conv_bwd_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t K) {
    return sizeof(float) * (size_t)(bwd_rows(bwd_shape(B, T, C), B) * C * (K + 1));
}

int64_t conv_workgroups(int64_t B, int64_t T, int64_t C) {
    const Shape s = fwd_shape(B, T, C);
    return s.ncb * B * s.nunit;
}

hipError_t launch_conv_fwd(const ConvArgs& a) {
    const Shape s = fwd_shape(a.B, a.T, a.C);
    const dim3 grid((unsigned)(s.ncb * s.nunit * a.B));
    if (a.K == 4) fwd_t<4>(a, grid, s);
    else if (a.K == 3) fwd_t<3>(a, grid, s);
    else fwd_t<2>(a, grid, s);
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvArgs& a) {
    const int64_t ncg = cdiv(a.C, 4);
    const dim3 grid((unsigned)cdiv(a.B * ncg, 256));
    if (a.K == 4) step_t<4>(a, grid, ncg);
    else if (a.K == 3) step_t<3>(a, grid, ncg);
    else step_t<2>(a, grid, ncg);
    return hipGetLastError();
}

hipError_t launch_conv_bwd(const ConvArgs& a) {
    const Shape s = bwd_shape(a.B, a.T, a.C);
    const int64_t nrow = bwd_rows(s, a.B);
    const dim3 grid((unsigned)(s.ncb * nrow));
    if (a.K == 4) bwd_k<4>(a, grid, s, nrow);
    else if (a.K == 3) bwd_k<3>(a, grid, s, nrow);
    else bwd_k<2>(a, grid, s, nrow);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    return launch_sum_partials(a.part, nrow, a.C * (a.K + 1), a.dw, a.C * a.K, a.dbias,
                               a.stream);
}

}  // namespace gdr
