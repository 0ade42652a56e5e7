// gdr_linear_attn_fwd / _bwd: linear attention with a decay per head,
//
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = s S_t q_t,
//
// in chunks of C tokens.  With L the running sum of g inside a chunk,
//
//   P_ij = s (q_i . k_j) e^{L_i - L_j}  (j <= i),
//   o_i  = sum_j P_ij v_j + s e^{L_i} S q_i,
//   S'   = e^{L_C} S + sum_j e^{L_C - L_j} v_j k_j^T.
//
// The backward is the same chain three times, with the tensors in other places
// (G_t the gradient of S_t, carried backwards in time):
//
//   dq_i = s sum_{j <= i} e^{L_i - L_j} (do_i . v_j) k_j + ..      from S^T, forwards
//   dk_j = s sum_{i >= j} e^{L_i - L_j} (do_i . v_j) q_i + ..      from G^T, backwards
//   dv_j = s sum_{i >= j} e^{L_i - L_j} (q_i . k_j) do_i + ..      from G, backwards
//
// and the decay's gradient is what the exponents of all pairs around a token say:
// dg_t = sum_{i >= t} (q_i . dq_i - k_i . dk_i) + <dS_T, S_T>.
//
// A workgroup of 16 waves follows one (sequence, head) for 64 of the out channels, in
// three teams (a wave of U and L and two of O to a SIMD) and two stages a chunk:
//
//   L (4 waves)  brings tiles: chunk n to LDS in stage 1; it asks for chunk n + 2 in
//                both (40 KB at once would be more than a compute unit has in flight)
//   U (4 waves)  carries the state: S through chunk n - 1, then S to LDS
//   O (8 waves)  forms the out: out of chunk n - 1, then P of chunk n; one of its waves
//                the factors of chunk n + 1
//
// Wave w of U keeps channels 16 w .. 16 w + 15 of the state in registers, transposed, in
// the layout of a product's result, which is also that of the next product's operand.
//
// Bound by the two stages' chains of dependent steps between the barriers; no unit is
// full.  bf16 B8 T4096, 16 heads of 128, bf16 out: 256 workgroups, 175 us (3.1 TB/s), 5300
// cycles a chunk at the 1.95 GHz (of 2.4) that the chip holds under many such calls (155
// us at 2.4, calls apart).  A chunk has 408 products of 16 cycles to a compute unit (40 P,
// 48 and 128 out, 192 the state in three terms): 1632 cycles on each SIMD, 31 %; its
// vector instructions take 2250 (42 %), LDS 2950 (56 %, 500 of them bank conflicts).
// Without loads and stores it would be 160 us.  Four waves, each with all the parts, took
// 454.
//
// The backward (B4: 344 us) alike: dq and dk in one launch, 217 to 227, with three terms
// everywhere for the decay's gradient (7300 cycles a chunk, matrix 27 %, vector 44 %, LDS
// 53 %), dv in another, 83 to 87 (5500 cycles, matrix 30 %), the decay 28.
#include <type_traits>

#include "linear_chain.h"

namespace gdr {
namespace la {
namespace {

template <class P, int KD> struct Shared {
    typename P::T x[2][P::C * KD], y[2][P::C * KD], z[2][P::C * ZB];
    typename P::T p[P::NO][PTile<P>::SIZE];
    typename P::T h[P::NO][ZB * KD];        // the state's terms, rows of z's channels
    // factors of the running log decay: from the chunk's start, to its end
    float enter[2][P::C], leave[2][P::C], total[2];
    int bad[2];             // 1 + the last chunk with a z that is no number
    // the running log decay (base 2) in two terms
    float lh[2][P::C], ll[2][P::C];
};

// What the states alone need of it, for NZ blocks of z's channels.
template <class P, int KD, int NZ> struct StatesShared {
    typename P::T y[2][P::C * KD], z[2][NZ * P::C * ZB];
    float leave[2][P::C], total[2];
};

// Tile (i, j) of P^T (row 4 g + r: token j, column m: token i) and its operands, which
// are read a tile ahead of their use.
template <class P, int KD> struct PTileWork {
    static constexpr int NK = KD / 32;
    typename P::Frag xf[NK], yf[NK];
    typename Tile<P, KD, ROWS>::Rows x;
    typename Tile<P, KD, BOTH>::Rows y;
    __device__ __forceinline__ void init(int lane) {
        x.init(lane);
        y.init(lane);
    }
    __device__ __forceinline__ void read(const Shared<P, KD>& s, int pb, int i, int j) {
        x.of(s.x[pb] + 16 * i * KD);
        y.of(s.y[pb] + 16 * j * KD);
        if constexpr (P::is_bf16) {         // fp32: too many registers
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                xf[k] = x.get(0, k);
                yf[k] = y.get(0, k);
            }
        }
    }
    __device__ __forceinline__ f32x4 product() {
        f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            if constexpr (!P::is_bf16) {
                xf[k] = x.get(0, k);
                yf[k] = y.get(0, k);
            }
            c = P::mma(yf[k], xf[k], c);
        }
        return c;
    }
    __device__ __forceinline__ void write(Shared<P, KD>& s, int pb, int i, int j, int lane,
                                          float scale, const f32x4& c) {
        const int g = lane >> 4, m = lane & 15;
        const float lh = s.lh[pb][16 * i + m], ll = s.ll[pb][16 * i + m];
        const f32x4 jh = *reinterpret_cast<const f32x4*>(&s.lh[pb][16 * j + 4 * g]);
        const f32x4 jl = *reinterpret_cast<const f32x4*>(&s.ll[pb][16 * j + 4 * g]);
        const int past = 16 * (i - j) + m - 4 * g;      // tokens j on which i looks back
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v[r] = c[r] * (__builtin_amdgcn_exp2f((lh - jh[r]) + (ll - jl[r])) * scale);
            if (r > past) v[r] = 0.f;
        }
        typedef PTile<P> TP;
        const int to = TP::piece(m, ((j & 1) * 16 + 4 * g) / P::EP) + 4 * g % P::EP +
                       TP::tile(i, j);
        if constexpr (P::is_bf16) {
            uint32_t w0[P::NO], w1[P::NO];
            P::template split_pair<P::NO>(v[0], v[1], w0);
            P::template split_pair<P::NO>(v[2], v[3], w1);
#pragma unroll
            for (int q = 0; q < P::NO; ++q)
                *reinterpret_cast<uint2*>(s.p[q] + to) = uint2{w0[q], w1[q]};
        } else {
            *reinterpret_cast<f32x4*>(s.p[0] + to) = v;
        }
    }
};

// Team L: tiles of the chunks, from memory to LDS; of z, NZ blocks of channels.
template <class P, int KD, bool OUT, int NZ> struct Bringer {
    typedef typename P::T T;
    // what is on its way for one chunk
    struct Coming {
        Stage<P, KD, ROWS> x;
        Stage<P, KD, BOTH> y;
        Stage<P, ZB, BOTH> z[NZ];
    };
    const char *xb, *yb, *zb;
    int64_t xt, yt, zt;
    bool back;

    __device__ __forceinline__ Bringer(const Place& at, const LaJob& jb, int tid, Coming& c)
        : back(jb.back) {
        xb = OUT ? static_cast<const char*>(head_base(jb.x, at.b, at.h, sizeof(T))) : nullptr;
        yb = static_cast<const char*>(head_base(jb.y, at.b, at.h, sizeof(T)));
        zb = static_cast<const char*>(head_base(jb.z, at.b, at.h, sizeof(T))) +
             at.zb * NZ * ZB * sizeof(T);
        xt = jb.x.st;
        yt = jb.y.st;
        zt = jb.z.st;
        if constexpr (OUT) c.x.init(tid, jb.kd, xt, back);
        c.y.init(tid, jb.kd, yt, back);
#pragma unroll
        for (int i = 0; i < NZ; ++i) c.z[i].init(tid, jb.zd - (at.zb * NZ + i) * ZB, zt, back);
    }
    __device__ __forceinline__ void ask_x(int64_t t0, int len, Coming& c) {
        if constexpr (OUT) c.x.load(xb + t0 * xt * (int)sizeof(T), xt, len, back);
    }
    __device__ __forceinline__ void ask_yz(int64_t t0, int len, Coming& c) {
        c.y.load(yb + t0 * yt * (int)sizeof(T), yt, len, back);
#pragma unroll
        for (int i = 0; i < NZ; ++i)
            c.z[i].load(zb + (t0 * zt + i * ZB) * (int)sizeof(T), zt, len, back);
    }
    template <class S> __device__ __forceinline__ void put_yz(S& s, int64_t n, int len, Coming& c) {
        const int buf = (int)(n & 1);
        c.y.put(s.y[buf], len);
#pragma unroll
        for (int i = 0; i < NZ; ++i) c.z[i].put(s.z[buf] + i * P::C * ZB, len);
        if constexpr (OUT) {
            if (c.z[0].bad()) s.bad[buf] = (int)(n + 1);
        }
    }
};

// The factors of the chunks' decays, by one wave.
template <class P, bool OUT> struct Decays {
    static constexpr int C = P::C;
    const LaChain& a;
    const Place& at;
    int lane;
    float inter, upd;
    bool back;
    float next;                     // the lane's log decay of the chunk to be scanned next
    double run;

    __device__ __forceinline__ Decays(const LaChain& a_, const Place& at_, const LaJob& jb,
                                      int lane_)
        : a(a_), at(at_), lane(lane_), inter(jb.inter), upd(jb.upd), back(jb.back), next(0.f),
          run(0.0) {}
    __device__ __forceinline__ void ask(int64_t t0, int len) {
        next = 0.f;
        if (lane < len) next = decay_of(a, at.b, at.h, back ? t0 + len - lane : t0 + lane);
    }
    // Factors of chunk n.  Running sums are in 64 bits: behind a reset, the differences
    // of sums far larger than themselves decide the factors.
    template <class S> __device__ __forceinline__ void scan(S& s, int64_t n) {
        const int buf = (int)(n & 1);
        const double l = wave_scan64(base2(next)), end = lane64(l, C - 1);
        if (lane < C) {
            if constexpr (OUT) {
                s.lh[buf][lane] = (float)l;
                s.ll[buf][lane] = (float)(l - (double)(float)l);
                s.enter[buf][lane] = inter * __builtin_amdgcn_exp2f((float)l);
            }
            s.leave[buf][lane] = upd * __builtin_amdgcn_exp2f((float)(end - l));
        }
        if (lane == 0) s.total[buf] = __builtin_amdgcn_exp2f((float)end);
        run += end;
    }
};

// Team U: the state of 16 channels of z per wave, transposed: row 4 g + r of tile u is
// channel 16 u + 4 g + r of x and y, column m channel zc + m of z.
template <class P, int KD> struct State {
    typedef Tile<P, KD, BOTH> TY;
    typedef Tile<P, ZB, BOTH> TZ;
    static constexpr int NU = KD / 16, NJ = P::C / 32;
    f32x4 H[NU];
    int g, m, w, zc, zd, kd;
    int64_t hz, hk;
    typename TY::Cols cols;
    typename TZ::Cols zcol;
    uint32_t ho;                    // the wave's part of the terms in LDS

    // of z's channels from `first` on
    __device__ __forceinline__ State(const LaJob& jb, int first, int tid) {
        const int lane = tid & 63;
        w = __builtin_amdgcn_readfirstlane(tid >> 6);
        g = lane >> 4;
        m = lane & 15;
        zc = first + 16 * w;
        zd = jb.zd;
        kd = jb.kd;
        hz = jb.hz;
        hk = jb.hk;
        cols.init(lane);
        zcol.init(lane, w % 4);
#pragma unroll
        for (int u = 0; u < NU; ++u) H[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ bool has(int u) const {
        return zc + m < zd && 16 * u + 4 * g < kd;
    }
    // The lane's first element of the state in memory.  Formed anew where it is used:
    // all the offsets, kept over the loop, would not leave registers for the rest.
    __device__ __forceinline__ int first() const {
        int e = (zc + m) * (int)hz + 4 * g * (int)hk;
        asm volatile("" : "+v"(e));
        return e;
    }
    __device__ __forceinline__ void load(const float* p) {
        p += first();
        if (hk == 1) {
#pragma unroll
            for (int u = 0; u < NU; ++u)
                if (has(u)) H[u] = *reinterpret_cast<const f32x4_e4*>(p + 16 * u);
            return;
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
            if (has(u)) {
#pragma unroll
                for (int r = 0; r < 4; ++r) H[u][r] = p[(16 * u + r) * (int)hk];
            }
    }
    __device__ __forceinline__ void store(float* p, float f) const {
        p += first();
        if (hk == 1) {
#pragma unroll
            for (int u = 0; u < NU; ++u)
                if (has(u)) *reinterpret_cast<f32x4_e4*>(p + 16 * u) = H[u] * f;
            return;
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
            if (has(u)) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    p[(16 * u + r) * (int)hk] = H[u][r] * f;
            }
    }
    // through the chunk in `buf`
    template <class S> __device__ __forceinline__ void move(const S& s, int buf) {
        cols.of(s.y[buf]);
        zcol.of(s.z[buf] + w / 4 * (P::C * ZB));
        // four tiles (fp32: two) at a time, the next ones' operands on their way: more
        // would not fit the registers, and a spill waits behind L's loads
        constexpr int W = P::is_bf16 ? 4 : 2, PER = NU / W, NG = NJ * PER;
        typename P::Frag yf[2][W], z[NJ];
        f32x4 l[NJ][2];
        auto fetch = [&](int i) {
#pragma unroll
            for (int e = 0; e < W; ++e) yf[i & 1][e] = cols.get(i / PER, i % PER * W + e);
        };
        const float tot = s.total[buf];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            z[j] = zcol.get(j, 0);
            l[j][0] = *reinterpret_cast<const f32x4*>(&s.leave[buf][32 * j + 8 * g]);
            l[j][1] = *reinterpret_cast<const f32x4*>(&s.leave[buf][32 * j + 8 * g + 4]);
        }
        fetch(0);
#pragma unroll
        for (int u = 0; u < NU; ++u) H[u] *= tot;
        Terms<typename P::Frag, P::NS> zt;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            if (i % PER == 0) {             // z scaled to the chunk's end, as terms
                const int j = i / PER;
                f32x8 v = P::widen(z[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= l[j][e / 4][e % 4];
                P::template split<P::NS>(v, zt);
            }
            if (i + 1 < NG) fetch(i + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = P::NS - 1; q >= 0; --q)
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const int u = i % PER * W + e;
                    H[u] = P::mma(yf[i & 1][e], zt.t[q], H[u]);
                }
        }
    }
    // its terms to LDS, rows of z's channels: where, and all of it
    __device__ __forceinline__ void shows(const Shared<P, KD>& s) {
        ho = lds_at(s.h[0]) +
             (Tile<P, KD, ROWS>::at(m, 4 * g) + 16 * w * KD) * (uint32_t)sizeof(typename P::T);
    }
    __device__ __forceinline__ void show() {
        asm volatile("" : "+v"(ho));        // as in first()
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const uint32_t to = ho ^ (16 * u * (uint32_t)sizeof(typename P::T));
            if constexpr (P::is_bf16) {
                uint32_t w0[P::NO], w1[P::NO];
                P::template split_pair<P::NO>(H[u][0], H[u][1], w0);
                P::template split_pair<P::NO>(H[u][2], H[u][3], w1);
#pragma unroll
                for (int q = 0; q < P::NO; ++q)
                    lds_set(to, q * ZB * KD * 2, u32x2{w0[q], w1[q]});
            } else {
                lds_set(to, 0, H[u]);
            }
        }
    }
};

// Tokens [ta, tb) of a segment in chunks, in the chain's order.
struct Chunks {
    int64_t ta, tb, nc;
    int C;
    bool back;
    __device__ __forceinline__ Chunks(const LaChain& a, const Place& at, bool back_, int C_)
        : C(C_), back(back_) {
        ta = at.seg * a.L;
        tb = ta + a.L < a.T ? ta + a.L : a.T;
        nc = (tb - ta + C - 1) / C;
    }
    // chunk n: tokens t0 .. t0 + len - 1, rows from the first on (back: from the last)
    __device__ __forceinline__ void get(int64_t n, int64_t& t0, int& len) const {
        t0 = ta + (back ? nc - 1 - n : n) * C;
        len = (int)(tb - t0 < C ? tb - t0 : C);
    }
};

// The chain's out (and its states).  GRAD: jobs may have kept states and dots.
template <class P, int KD, bool GRAD>
__global__ __launch_bounds__(1024) void chain_kernel(LaChain a) {
    constexpr int C = P::C, NK = KD / 32, NI = C / 16, NT = NI / 2;
    typedef Tile<P, KD, ROWS> TX;
    typedef Tile<P, ZB, BOTH> TZ;
    typedef PTile<P> TP;
    typedef typename P::T T;
    extern __shared__ __attribute__((aligned(512))) char smem[];
    Shared<P, KD>& s = *reinterpret_cast<Shared<P, KD>*>(smem);

    Place at;
    if (!place(a, blockIdx.x, ZB, at)) return;
    const LaJob& jb = a.job[at.job];
    const Chunks ch(a, at, jb.back, C);
    const int64_t nc = ch.nc, bh = at.b * a.H + at.h;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool back = jb.back;

    // tiles above the diagonal stay 0
    for (int i = threadIdx.x; i < P::NO * TP::SIZE; i += 1024) (&s.p[0][0])[i] = 0;
    if (threadIdx.x < 2) s.bad[threadIdx.x] = 0;

    if (wv >= 12) {
        // ---- team L ----
        typedef Bringer<P, KD, true, 1> L;
        typename L::Coming even, odd;
        L l(at, jb, threadIdx.x - 768, even);
        odd = even;
        int64_t t0;
        int len;
        ch.get(0, t0, len);
        l.ask_x(t0, len, even);
        l.ask_yz(t0, len, even);
        if (nc > 1) {
            ch.get(1, t0, len);
            l.ask_x(t0, len, odd);
            l.ask_yz(t0, len, odd);
        }
        lds_barrier();
        auto turn = [&](int64_t n, typename L::Coming& c) {
            int64_t t0, t2 = 0;
            int len, len2 = 0;
            if (n + 2 < nc) ch.get(n + 2, t2, len2);
            if (n < nc) {
                ch.get(n, t0, len);
                c.x.put(s.x[n & 1], len);
                if (n + 2 < nc) l.ask_x(t2, len2, c);
                l.put_yz(s, n, len, c);
            }
            lds_barrier();
            if (n + 2 < nc) l.ask_yz(t2, len2, c);
            lds_barrier();
        };
        for (int64_t n = 0; n <= nc; n += 2) {
            turn(n, even);
            if (n + 1 <= nc) turn(n + 1, odd);
        }
        return;
    }
    if (wv >= 8) {
        // ---- team U ----
        State<P, KD> st(jb, at.zb * ZB, threadIdx.x - 512);
        st.shows(s);
        if (at.seg == (back ? a.nseg - 1 : 0)) {
            if (jb.h_in) st.load(jb.h_in + bh * a.state);
        } else {
            const int64_t slot = (at.seg + (back ? 1 : 0)) * jb.h_step - 1;
            st.load(jb.h_seg + (slot * a.B * a.H + bh) * a.state);
        }
        float* const keep = GRAD ? jb.keep : nullptr;
        lds_barrier();
        for (int64_t n = 0; n <= nc; ++n) {
            if (n > 0) st.move(s, (int)((n - 1) & 1));
            lds_barrier();
            if (n < nc) st.show();
            if (GRAD && keep && n > 0) {
                int64_t t0;
                int len;
                ch.get(n - 1, t0, len);
                const int64_t mark = back ? t0 : t0 + len;
                if (back ? (mark > 0 && mark % a.every == 0)
                         : (mark < a.T ? mark % a.every == 0 : jb.keep_end))
                    st.store(keep + (((mark + a.every - 1) / a.every - 1) * a.B * a.H + bh) *
                                        a.state, 1.f);
            }
            lds_barrier();
        }
        if (jb.h_out && at.seg == (back ? 0 : a.nseg - 1)) {
            float f = 1.f;
            if (jb.end_decay)
                f = __builtin_amdgcn_exp2f((float)base2(decay_of(a, at.b, at.h, 0)));
            st.store(jb.h_out + bh * a.state, f);
        }
        return;
    }

    // ---- team O: 16 channels of z (wave & 3), token tiles {0, 2} or {1, 3} (fp32: 0 or
    // 1), which are as many 32-deep contractions ----
    const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int zg = wv & 3, half = wv >> 2;
    auto tile = [&](int t) { return half + 2 * t; };
    typename TX::Rows xrow, hrow;
    typename TZ::Cols zcol;
    typename TP::Rows prow;
    PTileWork<P, KD> pw;
    xrow.init(lane);
    hrow.init(lane);
    hrow.of(s.h[0] + 16 * zg * KD);
    zcol.init(lane, zg);
    prow.init(lane, s.p[0] + TP::tile(half, 0));
    pw.init(lane);
    const int zd = jb.zd, zc = at.zb * ZB + 16 * zg;
    const bool mine = zc + 4 * g < zd;                  // whether the lane has out channels
    const bool out16 = jb.out_bf16;
    const size_t oe = out16 ? 2 : 4;
    const uint32_t ot = (uint32_t)(jb.ot * (int64_t)oe);
    char* ob = static_cast<char*>(jb.out) + (at.b * jb.ob + at.h * jb.oh + zc + 4 * g) * oe;
    const bool dots = GRAD && jb.dots;
    const char* rb = dots ? static_cast<const char*>(head_base(jb.r, at.b, at.h, sizeof(T))) +
                                (zc + 4 * g) * sizeof(T)
                          : nullptr;
    const uint32_t rt = dots ? (uint32_t)(jb.r.st * sizeof(T)) : 0u;
    float* const db = dots ? jb.dots + (((int64_t)(zc >> 4) * a.B + at.b) * a.H + at.h) * a.T
                           : nullptr;
    // the wave's tiles of P, at most two: of the ten in bf16, of the three in fp32.
    // Wave 3 has none: the factors are its part
    const int pi = NI == 4 ? (0x32130233 >> (4 * wv)) & 3 : (wv == 1 ? 0 : 1);
    const int pj = NI == 4 ? (0x32020010 >> (4 * wv)) & 3 : (wv == 2 ? 1 : 0);
    const int qi = wv, qj = wv == 2 ? 1 : wv;
    const int np = NI == 4 ? (wv < 3 ? 2 : wv == 3 ? 0 : 1) : (wv < 3 ? 1 : 0);
    const float pair = jb.pair;
    Decays<P, true> dec(a, at, jb, lane);
    if (wv == 3) {
        int64_t t0;
        int len;
        ch.get(0, t0, len);
        dec.ask(t0, len);
        dec.scan(s, 0);
        if (nc > 1) {
            ch.get(1, t0, len);
            dec.ask(t0, len);
        }
    }

    lds_barrier();
    for (int64_t n = 0; n <= nc; ++n) {
        f32x4 O[NT];
        int64_t t0 = 0;
        int len = 0;
        Row<4, P::is_bf16, false> rr[GRAD ? NT : 1];
        if (n > 0) {
            const int buf = (int)((n - 1) & 1);
            ch.get(n - 1, t0, len);
            if constexpr (GRAD) {
                if (dots) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        int row = 16 * tile(t) + m;
                        row = row < len ? row : len - 1;
                        rr[t].load(rb + t0 * jb.r.st * (int)sizeof(T) +
                                       (back ? len - 1 - row : row) * rt, 0, mine ? 4 : 0);
                    }
                }
            }
            // out^T (row 4 g + r: channel, column m: token) from the start state
            typename P::Frag xf[2][NT], hf[2][P::NO];
            xrow.of(s.x[buf] + 16 * half * KD);
            hrow.fresh();
            auto fetch = [&](int k) {
#pragma unroll
                for (int t = 0; t < NT; ++t) xf[k & 1][t] = xrow.get(2 * t, k);
#pragma unroll
                for (int q = 0; q < P::NO; ++q) hf[k & 1][q] = hrow.get(ZB / 16 * q, k);
            };
#pragma unroll
            for (int t = 0; t < NT; ++t) O[t] = f32x4{0.f, 0.f, 0.f, 0.f};
            fetch(0);
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if (k + 1 < NK) fetch(k + 1);
#pragma unroll
                for (int q = P::NO - 1; q >= 0; --q)
#pragma unroll
                    for (int t = 0; t < NT; ++t) O[t] = P::mma(hf[k & 1][q], xf[k & 1][t], O[t]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) O[t] *= s.enter[buf][16 * tile(t) + m];
            if (__builtin_expect(s.bad[buf] != (int)n, 1)) {
                zcol.of(s.z[buf]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const typename P::Frag zf = zcol.get(j, 0);
#pragma unroll
                    for (int q = P::NO - 1; q >= 0; --q)
#pragma unroll
                        for (int t = j; t < NT; ++t)
                            O[t] = P::mma(zf, prow.get(q * TP::SIZE, 2 * t, j), O[t]);
                }
            } else {
                // a value of z that is no number must not meet the zeros of the tokens
                // before it: one by one
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int i = 16 * tile(t) + m;
                    for (int j = 0; j <= i; ++j) {
                        float pv = 0.f;
#pragma unroll
                        for (int q = P::NO - 1; q >= 0; --q) {
                            const T w = s.p[q][TP::at(i, j)];
                            if constexpr (P::is_bf16) pv += bf2f(w);
                            else pv += w;
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const T w = s.z[buf][TZ::at(j, 16 * zg + 4 * g + r)];
                            float zv;
                            if constexpr (P::is_bf16) zv = bf2f(w);
                            else zv = w;
                            O[t][r] = __builtin_fmaf(pv, zv, O[t][r]);
                        }
                    }
                }
            }
        }
        lds_barrier();
        // before the stores: the wait for the decays would be one for these too
        if (wv == 3 && n + 1 < nc) {
            dec.scan(s, n + 1);
            if (n + 2 < nc) {
                int64_t t2;
                int len2;
                ch.get(n + 2, t2, len2);
                dec.ask(t2, len2);
            }
        }
        const int nb = (int)(n & 1);
        if (n < nc && np > 0) pw.read(s, nb, pi, pj);
        if (n > 0) {
            if constexpr (GRAD) {
                if (dots) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const int row = 16 * tile(t) + m;
                        // in 64 bits, rounded once: what cancels between channels, and
                        // then between q . dq and k . dk, is not lost (3 us of 344)
                        float rv[4];
                        double d = 0.0;
                        rr[t].unpack(rv);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            d = __builtin_fma((double)rv[r], (double)O[t][r], d);
                        d += __shfl_xor(d, 16, 64);
                        d += __shfl_xor(d, 32, 64);
                        if (g == 0 && row < len && zc < zd)
                            db[t0 + (back ? len - 1 - row : row)] = (float)d;
                    }
                }
            }
            char* oc = ob + t0 * ot;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int row = 16 * tile(t) + m;
                if (mine && row < len) {
                    const uint32_t off = (uint32_t)(back ? len - 1 - row : row) * ot;
                    if (out16)
                        *reinterpret_cast<u32x2_e2*>(oc + off) =
                            u32x2_e2{cvt_pk(O[t][0], O[t][1]), cvt_pk(O[t][2], O[t][3])};
                    else
                        *reinterpret_cast<f32x4_e4*>(oc + off) = O[t];
                }
            }
        }
        if (n < nc && np > 0) {
            f32x4 c = pw.product();
            if (np > 1) {
                pw.read(s, nb, qi, qj);
                pw.write(s, nb, pi, pj, lane, pair, c);
                c = pw.product();
                pw.write(s, nb, qi, qj, lane, pair, c);
            } else {
                pw.write(s, nb, pi, pj, lane, pair, c);
            }
        }
        lds_barrier();
    }
}

// The states at the segments' ends alone, and the segments' decays.  A workgroup has up
// to 128 channels of z, so that y is read once and segments can be half as long: 72 us
// and 9 to compose them where 64 channels took 92 and 6 (B1 T32768 H16, heads of 128;
// 250 MB of k and v).  Bound by the state's products and terms: 50 us without.
template <class P, int KD, int NZ>
__global__ __launch_bounds__(256 + 256 * NZ) void states_kernel(LaChain a) {
    __shared__ __attribute__((aligned(512))) StatesShared<P, KD, NZ> s;
    Place at;
    if (!place(a, blockIdx.x, NZ * ZB, at)) return;
    const LaJob& jb = a.job[at.job];
    if (at.seg == (jb.back ? 0 : a.nseg - 1)) return;       // no segment behind it
    const Chunks ch(a, at, jb.back, P::C);
    const int64_t nc = ch.nc;
    const int64_t to = (at.seg - (jb.back ? 1 : 0)) * a.B * a.H + at.b * a.H + at.h;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wv >= 4 * NZ) {
        typedef Bringer<P, KD, false, NZ> L;
        typename L::Coming even, odd;
        L l(at, jb, threadIdx.x - 256 * NZ, even);
        odd = even;
        Decays<P, false> dec(a, at, jb, threadIdx.x & 63);
        int64_t t0;
        int len;
        ch.get(0, t0, len);
        if (wv == 4 * NZ + 3) dec.ask(t0, len);
        l.ask_yz(t0, len, even);
        if (nc > 1) {
            ch.get(1, t0, len);
            l.ask_yz(t0, len, odd);
        }
        auto turn = [&](int64_t n, typename L::Coming& c) {
            int64_t t0;
            int len;
            if (wv == 4 * NZ + 3) {
                dec.scan(s, n);
                if (n + 1 < nc) {
                    ch.get(n + 1, t0, len);
                    dec.ask(t0, len);
                }
            }
            ch.get(n, t0, len);
            l.put_yz(s, n, len, c);
            if (n + 2 < nc) {
                ch.get(n + 2, t0, len);
                l.ask_yz(t0, len, c);
            }
            lds_barrier();
        };
        for (int64_t n = 0; n < nc; n += 2) {
            turn(n, even);
            if (n + 1 < nc) turn(n + 1, odd);
        }
        lds_barrier();              // U's last chunk
        if (at.zb == 0 && threadIdx.x == 256 * NZ + 192)
            jb.seg_decay[to] = __builtin_amdgcn_exp2f((float)dec.run);
        return;
    }
    State<P, KD> st(jb, at.zb * NZ * ZB, threadIdx.x);
    lds_barrier();
    for (int64_t n = 0; n < nc; ++n) {
        st.move(s, (int)(n & 1));
        lds_barrier();
    }
    st.store(jb.h_out + to * a.state, 1.f);
}

// States at the marks between segments, in place, from the segments' own (as from a
// start of zeros): at(next) = decay at(this) + own.  Up to two chains at once.  `copy`
// (or NULL) receives the state that they start from.
struct Compose {
    int64_t BH, state, marks;
    float* buf[2];
    const float *decay[2], *h0[2];
    float* copy[2];
    bool back[2];
};

__global__ __launch_bounds__(256) void compose_kernel(Compose a) {
    constexpr int N = 16;
    const int k = blockIdx.y;
    const int64_t n = a.BH * a.state, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float* buf = a.buf[k] + i;
    const float* decay = a.decay[k] + i / a.state;
    float h = a.h0[k] ? a.h0[k][i] : 0.f;
    if (a.copy[k]) a.copy[k][i] = h;
    const bool back = a.back[k];
    // batches of loads: a store would hold back the next segment's
    for (int64_t c = 0; c < a.marks; c += N) {
        float own[N], d[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t p = back ? a.marks - 1 - c - e : c + e;
            own[e] = d[e] = 0.f;
            if (c + e < a.marks) {
                own[e] = buf[p * n];
                d[e] = decay[p * a.BH];
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t p = back ? a.marks - 1 - c - e : c + e;
            h = d[e] * h + own[e];
            if (c + e < a.marks) buf[p * n] = h;
        }
    }
}

// Sums over the heads that share one: part [rows, Hk, share, D] to out [rows, Hk, D],
// for dq and dk at once.
struct Share {
    const float* part[2];
    void* out[2];
    bool bf16;
    int64_t n, share, D;
};

// Workgroup `id` of `count`, of dq (side 0) or dk.
__device__ __forceinline__ void share_heads(const Share& a, int side, int64_t id, int64_t count) {
    const float* part = a.part[side];
    for (int64_t i = id * 256 + threadIdx.x; i < a.n; i += count * 256) {
        const int64_t row = i / (a.D / 4), c = i % (a.D / 4) * 4;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        for (int64_t k = 0; k < a.share; ++k)
            x += *reinterpret_cast<const f32x4*>(part + (row * a.share + k) * a.D + c);
        const float v[4] = {x[0], x[1], x[2], x[3]};
        row_store<4, false>(a.out[side], row * a.D + c, a.bf16, v, 4);
    }
}

constexpr int kMostKept = 512, kTurns = kMostKept / 256;   // tokens between kept states

struct DecayGrad {
    int64_t B, T, H, every, nblk, state;
    int nq;                         // slots of either sum
    const float *q, *k;             // [nq][B][H][T] sums of q . dq and k . dk
    const float *skeep, *gkeep;     // states after, gradients before each block's end
    const float *ds_final, *s0;
    const float* g;
    bool g_head;
    float* dg;                      // [B, T, H], or per head:
    double* part;                   // [B nblk][H]
};

// wave_scan64 in runs: sums from a lane's run's first lane on (`from`; -1: it began in a
// wave before).  Steps from before it are left out, whatever they hold.
template <class V> __device__ __forceinline__ V run_scan(V x, int lane, int from) {
    auto move = [](V v, auto ctrl, auto rows) -> V {
        if constexpr (sizeof(V) == 8) return dpp_mov64<ctrl.value, rows.value>(v);
        else return dpp_mov<ctrl.value, rows.value>(v);
    };
    auto step = [&](auto ctrl, auto rows, bool within) {
        const V y = move(x, ctrl, rows);
        x += within ? y : V(0);
    };
    typedef std::integral_constant<int, 0xF> all;
    step(std::integral_constant<int, 0x111>(), all(), lane - 1 >= from);
    step(std::integral_constant<int, 0x112>(), all(), lane - 2 >= from);
    step(std::integral_constant<int, 0x114>(), all(), lane - 4 >= from);
    step(std::integral_constant<int, 0x118>(), all(), lane - 8 >= from);
    step(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xA>(),
         from < (lane & 48));
    step(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xC>(), from < 32);
    return x;
}

// dg of one block of tokens of a (sequence, head): what all pairs across its end say,
// <G, S> there, and the running sum of q . dq - k . dk from the end, in 64 bits.  No pair
// lies across a decay of 0: such tokens cut a block into runs, each with a sum of its own,
// so that nothing of one packed sequence reaches another.
//
// The terms carry the roundings of dq and dk, so the sum's error grows with the distance
// from the end.  At a run's start the pairs across say what the whole run should sum up
// to: 0 at such a token, <G, S> at the block's start.  The difference is taken out in
// proportion to the sum of |q . dq| + |k . dk| from the end on, which is what the
// roundings in it are in proportion to: a token loses no more than its own terms may be
// off, however large others of the run are.  (In proportion to the distance, tokens 100
// times as large as those behind them left these with nothing but error.)
//
// That, the blocks' length and dots in 64 bits (chain_kernel) keep dg as exact as a form in
// fp32: bf16 B50 T2737 H1 32 x 128, ten draws, 0.38e-6 off on average and 0.9e-6 at most
// (fp32 0.38e-6 and 0.7e-6; with dots in fp32 0.51e-6 and 1.4e-6; one draw that was 2.0e-6
// with blocks of 1024 tokens from the end alone was 1.0e-6 from both ends of 512).  A sum
// per head, which adds all of them up, has blocks of 256: B2 T4109 H4 64 x 64 0.43e-6 and
// 1.3e-6 (0.28e-6 and 0.6e-6).  At B4 T4096 H16 of 128 (328 us with 1024) 512 cost 14 us,
// 256 30.
__device__ __forceinline__ void decay_grad(const DecayGrad& a, int64_t id) {
    __shared__ double red[4], part[kTurns][4];
    __shared__ float weight[kTurns][4], rate_off[kMostKept];
    __shared__ uint64_t first[kTurns][4];
    const int64_t h = id % a.H, b = id / a.H % a.B, p = id / a.H / a.B;
    const int64_t bh = b * a.H + h;
    const int tid = threadIdx.x;
    const int64_t t0 = p * a.every, t1 = t0 + a.every < a.T ? t0 + a.every : a.T;
    auto rate = [&](int64_t t) {
        const float g = a.g_head ? a.g[h] : a.g[(b * a.T + t) * a.H + h];
        return g < kLeast ? kLeast : g;
    };
    auto cuts = [&](int64_t t) { return rate(t) < -104.f; };        // e^g is 0
    // the pairs across the end of block o
    auto across = [&](int64_t o) {
        const bool last = o + 1 == a.nblk;
        const int64_t t = (o + 1) * a.every;
        const float* G = !last ? (cuts(t) ? nullptr : a.gkeep + (o * a.B * a.H + bh) * a.state)
                         : a.ds_final ? a.ds_final + bh * a.state : nullptr;
        double sum = 0.0;
        if (G) {
            const float* S = a.skeep + (o * a.B * a.H + bh) * a.state;
            // the state's size is a multiple of 64 floats, its place in the caller's
            // memory any
#pragma unroll 4
            for (int64_t i = 4 * tid; i < a.state; i += 1024) {
                const f32x4_e4 x = *reinterpret_cast<const f32x4_e4*>(G + i);
                const f32x4 y = *reinterpret_cast<const f32x4*>(S + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += (double)x[e] * (double)y[e];
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, 64);
        if ((tid & 63) == 0) red[tid >> 6] = sum;
        __syncthreads();
        sum = (red[0] + red[1]) + (red[2] + red[3]);
        __syncthreads();
        return last || !G ? sum : sum * (double)__builtin_amdgcn_exp2f(rate(t) * kLog2e);
    };
    // thread 0: the last token of 256 each
    const int wv = tid >> 6, lane = tid & 63;
    const int64_t n = a.B * a.H * a.T, row = bh * a.T;
    double e[kTurns];
    float w[kTurns];
    bool ends[kTurns];              // the run ends here: the token before has another sum
    int from[kTurns], run[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int64_t t = t1 - 1 - 256 * k - tid;
        e[k] = 0.0;
        w[k] = 0.f;
        ends[k] = false;
        bool begins = false;
        if (t >= t0) {
            // all loads at once, without branches between them
            float x[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t o = (i < a.nq ? i : 0) * n + row + t;
                x[2 * i] = a.q[o];
                x[2 * i + 1] = a.k[o];
            }
            ends[k] = cuts(t);
            begins = t + 1 < t1 && cuts(t + 1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                e[k] += i < a.nq ? (double)x[2 * i] - (double)x[2 * i + 1] : 0.0;
                w[k] += i < a.nq ? fabsf(x[2 * i]) + fabsf(x[2 * i + 1]) : 0.f;
            }
        }
        const uint64_t heads = __ballot(begins), upto = heads & (~0ull >> (63 - lane));
        from[k] = 63 - __clzll((long long)upto);
        run[k] = __popcll(upto);
        e[k] = run_scan(e[k], lane, from[k]);
        w[k] = run_scan(w[k], lane, from[k]);
        if (lane == 63) {
            part[k][wv] = e[k];
            weight[k][wv] = w[k];
            first[k][wv] = heads;
        }
    }
    const double tail = across(p);                      // part is there behind its barriers
    const double head = p > 0 ? across(p - 1) : 0.0;
    double carry = tail, sum = 0.0;
    float carried = 0.f;
    int runs = 0;
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (v == wv) {
                if (from[k] < 0) {
                    e[k] += carry;
                    w[k] += carried;
                }
                run[k] += runs;
            }
            const uint64_t heads = first[k][v];
            carry = heads ? part[k][v] : carry + part[k][v];
            carried = heads ? weight[k][v] : carried + weight[k][v];
            runs += __popcll(heads);
        }
    }
    // what a run's sum is off, for its weight.  The start state's own gradient is not
    // kept: then the end alone counts, as where something is no number
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int64_t t = t1 - 1 - 256 * k - tid;
        if (t < t0 || !(ends[k] || t == t0)) continue;
        double off = 0.0;
        if (ends[k]) off = e[k];
        else if (p > 0 || !a.s0) off = e[k] - head;
        const float r = (float)(off / (double)w[k]);
        rate_off[run[k]] = r - r == 0.f ? r : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int64_t t = t1 - 1 - 256 * k - tid;
        if (t < t0) continue;
        // a decay of 0 has no gradient
        const float r = rate_off[run[k]];
        const double d = ends[k] ? 0.0 : r != 0.f ? e[k] - (double)r * (double)w[k] : e[k];
        sum += d;
        if (a.dg) a.dg[(b * a.T + t) * a.H + h] = (float)d;
    }
    if (a.part) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, 64);
        if ((tid & 63) == 0) red[tid >> 6] = sum;
        __syncthreads();
        if (tid == 0) a.part[(b * a.nblk + p) * a.H + h] = (red[0] + red[1]) + (red[2] + red[3]);
    }
}

// What is left behind the chains: the decay's gradient by the first `decays` workgroups,
// the sums over shared heads by the others, side by side (a launch of its own for
// either cost 4 us more).
__global__ __launch_bounds__(256) void finish_kernel(DecayGrad d, Share m, uint32_t decays,
                                                     uint32_t shares) {
    if (blockIdx.x < decays) {
        decay_grad(d, blockIdx.x);
        return;
    }
    const uint32_t id = blockIdx.x - decays;
    share_heads(m, id < shares ? 0 : 1, id < shares ? id : id - shares, shares);
}

__global__ __launch_bounds__(64) void head_sum_kernel(const double* part, float* dg, int64_t n,
                                                      int64_t H) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 64) s += part[i * H + blockIdx.x];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d, 64);
    if (threadIdx.x == 0) dg[blockIdx.x] = (float)s;
}

// Workgroups of `width` channels of z.
template <class Fn>
hipError_t launch_one(Fn* fn, const LaChain& a, int width, int threads, size_t lds) {
    int64_t per = 0;
    for (int j = 0; j < a.njobs; ++j) per += (a.job[j].zd + width - 1) / width;
    const int64_t grid = (a.B * a.H * a.nseg + 7) / 8 * 8 * per;
    if (lds) {
        const hipError_t e = hipFuncSetAttribute(
            (const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(threads), lds, a.stream, a);
    return hipGetLastError();
}

template <class P, int KD> hipError_t launch_kd(const LaChain& a) {
    constexpr size_t lds = sizeof(Shared<P, KD>);
    static_assert(lds <= 160 * 1024, "LDS");
    for (int j = 0; j < a.njobs; ++j)
        if (a.job[j].keep || a.job[j].dots)
            return launch_one(chain_kernel<P, KD, true>, a, ZB, 1024, lds);
    return launch_one(chain_kernel<P, KD, false>, a, ZB, 1024, lds);
}

template <class P> hipError_t launch_chain_p(const LaChain& a) {
    return a.job[0].kd <= 64 ? launch_kd<P, 64>(a) : launch_kd<P, 128>(a);
}

// Jobs of one contraction width (all of a.job are on the same side of 64).
hipError_t launch_chain(const LaChain& a) {
    if (!a.bf16) return launch_chain_p<F32>(a);
    bool fine = false;          // whether an out is used in more than 16 bits
    for (int j = 0; j < a.njobs; ++j) fine |= a.job[j].out && (!a.job[j].out_bf16 || a.job[j].dots);
    return fine ? launch_chain_p<Bf16<3>>(a) : launch_chain_p<Bf16<2>>(a);
}

// The own end states of all segments but the last, of jobs of one contraction width and
// one width of z.
template <class P, int KD> hipError_t launch_states_kd(const LaChain& a) {
    if (a.job[0].zd <= ZB) return launch_one(states_kernel<P, KD, 1>, a, ZB, 512, 0);
    return launch_one(states_kernel<P, KD, 2>, a, 2 * ZB, 768, 0);
}

hipError_t launch_states(const LaChain& a) {
    if (!a.bf16)
        return a.job[0].kd <= 64 ? launch_states_kd<F32, 64>(a) : launch_states_kd<F32, 128>(a);
    return a.job[0].kd <= 64 ? launch_states_kd<Bf16<3>, 64>(a)
                             : launch_states_kd<Bf16<3>, 128>(a);
}

// Segments of L tokens; their start states at the marks between segments of Ls.
struct Plan {
    int64_t L, nseg, Ls, marks;
};

constexpr int kUnits = 256;         // compute units

int64_t blocks(int64_t d) { return (d + ZB - 1) / ZB; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t chunk(bool bf16) { return bf16 ? Bf16<3>::C : F32::C; }

// Segments: as many as fill the chip (a workgroup to each of 256 compute units), of at
// least two chunks.  A second pass over k and v and the states' round trip cost less
// than idle units: bf16 B1 T32768 H16, heads of 128, 386 us with 4 segments, 253 with 8;
// fp32 B3 T1025 H6 72 x 40 64 with 4, 33 with 11.
// `grain`: a segment's tokens are a multiple of it, or fewer.
Plan plan(int64_t T, int64_t units, bool bf16, int64_t grain) {
    const int64_t C = chunk(bf16), most = T / (2 * C);
    int64_t nseg = kUnits / units;
    if (nseg > most) nseg = most;
    if (nseg < 1) nseg = 1;
    int64_t L = cdiv(cdiv(T, nseg), C) * C;
    if (L > grain) L = cdiv(L, grain) * grain;
    nseg = cdiv(T, L);
    // two blocks of channels to a workgroup for the states alone: half segments
    const int64_t Ls = L % (2 * C) == 0 ? L / 2 : L;
    return {L, nseg, Ls, nseg > 1 ? cdiv(T, Ls) - 1 : 0};
}

Plan fwd_plan(int64_t B, int64_t T, int64_t H, int64_t Dv, bool bf16) {
    return plan(T, B * H * blocks(Dv), bf16, chunk(bf16));
}

// The backward's chains.  dq, dk and dv side by side, in segments p; or dq and dk first,
// and dv in segments pv that start where dk's chain has left states anyway.  With 64
// sequences and heads of 128 the first makes 384 workgroups, two rounds of the chip, the
// second 256 and then 256 of half the length: bf16 B4 T4096 H16 396 us and 324.
struct BwdPlan {
    Plan p, pv;
    bool apart;
    int64_t every, nblk;            // kept states: at whole numbers of `every` tokens
};

// Rounds of the chip times the chunks of a segment and what a workgroup's start costs.
double chain_cost(int64_t workgroups, int64_t L, bool bf16) {
    return (double)cdiv(workgroups, kUnits) * ((double)cdiv(L, chunk(bf16)) + 4.0);
}

BwdPlan bwd_plan(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, bool bf16,
                 bool g_head) {
    const int64_t most = g_head ? 256 : kMostKept;  // tokens between kept states (decay_grad)
    const int64_t BH = B * H, nk = BH * 2 * blocks(Dk), nv = BH * blocks(Dv);
    // a pass over the states alone takes half the time
    auto states = [&](const Plan& p) {
        return p.nseg > 1 ? 0.5 * chain_cost(p.marks * (nk / 2 + nv), p.Ls, bf16) + 4.0 : 0.0;
    };
    auto every = [&](const Plan& p) { return p.L > most ? most : p.L; };
    BwdPlan one{}, two{};
    one.p = plan(T, nk + nv, bf16, most);
    one.every = every(one.p);
    one.nblk = cdiv(T, one.every);
    two.p = plan(T, nk, bf16, most);
    two.apart = true;
    two.every = every(two.p);
    two.nblk = cdiv(T, two.every);
    double best = 0.0;
    for (int64_t n = 1; n <= two.nblk && n <= 64; ++n) {
        const int64_t L = cdiv(two.nblk, n) * two.every, nseg = cdiv(T, L);
        const double c = chain_cost(nv * nseg, L, bf16);
        if (n > 1 && c >= best) continue;
        best = c;
        two.pv = {L, nseg, L, 0};
    }
    if ((Dk <= 64) != (Dv <= 64)) return two;       // two launches in any case
    const double c1 = chain_cost((nk + nv) * one.p.nseg, one.p.L, bf16) + states(one.p);
    const double c2 = chain_cost(nk * two.p.nseg, two.p.L, bf16) + states(two.p) + best;
    return c2 < c1 ? two : one;
}

constexpr size_t up16(size_t n) { return (n + 15) / 16 * 16; }

LaJob job(const LaTensor& x, const LaTensor& y, const LaTensor& z, int64_t kd, int64_t zd) {
    LaJob j{};
    j.x = x;
    j.y = y;
    j.z = z;
    j.kd = (int)kd;
    j.zd = (int)zd;
    j.pair = j.inter = j.upd = 1.f;
    return j;
}

LaChain chain(const LaArgs& a, const Plan& p) {
    LaChain c{};
    c.B = a.B;
    c.T = a.T;
    c.H = a.H;
    c.L = p.L;
    c.nseg = p.nseg;
    c.bf16 = a.bf16;
    c.g = a.g;
    c.g_head = a.g_head;
    c.state = a.Dk * a.Dv;
    c.stream = a.stream;
    return c;
}

// Start states of the segments behind the first, of one or two jobs (h_in, hz and hk as
// for the whole chain), into buf, and the jobs set to start from them.  The first job
// starts from `copy`, where that is given.
hipError_t segment_states(LaChain c, const Plan& p, LaJob* const* jobs, int n, float* const* buf,
                          float* const* decay, float* copy) {
    Compose m{};
    m.BH = c.B * c.H;
    m.state = c.state;
    m.marks = p.marks;
    c.L = p.Ls;
    c.nseg = p.marks + 1;
    const bool both = n == 2 && (jobs[0]->kd <= 64) == (jobs[1]->kd <= 64);
    for (int i = 0; i < n; ++i) {
        LaJob j = *jobs[i];
        m.buf[i] = buf[i];
        m.decay[i] = decay[i];
        m.h0[i] = j.h_in;
        m.back[i] = j.back;
        jobs[i]->h_seg = buf[i];
        jobs[i]->h_step = p.L / p.Ls;
        j.h_out = buf[i];
        j.seg_decay = decay[i];
        c.job[both ? i : 0] = j;
        c.njobs = both ? 2 : 1;
        if (both && i == 0) continue;
        const hipError_t e = launch_states(c);
        if (e != hipSuccess) return e;
    }
    if (copy) {
        m.copy[0] = copy;
        jobs[0]->h_in = copy;
    }
    hipLaunchKernelGGL(compose_kernel, dim3((unsigned)cdiv(m.BH * m.state, 256), n), dim3(256), 0,
                       c.stream, m);
    return hipGetLastError();
}

}  // namespace
}  // namespace la

using namespace la;

// The largest launch of a call, in workgroups of 256.
int64_t la_fwd_workgroups(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, bool bf16) {
    const Plan p = fwd_plan(B, T, H, Dv, bf16);
    const int64_t chain = 4 * ((B * H * (p.marks + p.nseg) + 7) / 8 * 8 * blocks(Dv));
    const int64_t states = p.nseg > 1 ? cdiv(B * H * Dk * Dv, 256) : 0;
    return chain > states ? chain : states;
}

size_t la_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, bool bf16) {
    const Plan p = fwd_plan(B, T, H, Dv, bf16);
    if (p.nseg == 1) return 0;
    const size_t n = 4 * (size_t)(B * H), marks = (size_t)p.marks;
    return up16((marks + 1) * n * (size_t)(Dk * Dv)) + up16(marks * n);
}

hipError_t launch_la_fwd(const LaArgs& a) {
    const Plan p = fwd_plan(a.B, a.T, a.H, a.Dv, a.bf16);
    LaChain c = chain(a, p);
    LaJob j = job(a.q, a.k, a.v, a.Dk, a.Dv);
    j.pair = j.inter = a.scale;
    j.out = a.o;
    j.ob = a.T * a.H * a.Dv;
    j.ot = a.H * a.Dv;
    j.oh = a.Dv;
    j.out_bf16 = a.out_bf16;
    j.h_in = a.s0;
    j.hz = a.Dk;
    j.hk = 1;
    if (p.nseg > 1) {
        // in place, the last segment writes s0's memory while the first one may still have
        // to read it (nothing orders them in a launch): that starts from a copy
        float* buf = static_cast<float*>(a.workspace);
        float* const copy = buf + (size_t)(p.marks * a.B * a.H) * (size_t)c.state;
        float* decay = buf + up16(4 * (size_t)((p.marks + 1) * a.B * a.H) * (size_t)c.state) / 4;
        LaJob* const jobs[1] = {&j};
        const hipError_t e = segment_states(c, p, jobs, 1, &buf, &decay,
                                            a.s0 && a.s_final == a.s0 ? copy : nullptr);
        if (e != hipSuccess) return e;
    }
    j.h_out = a.s_final;
    c.njobs = 1;
    c.job[0] = j;
    return launch_chain(c);
}

namespace {

// Parts of the backward's workspace, in bytes from its start.
struct BwdSpace {
    size_t s, sdec, g, gdec, sk, gk, qd, kd, part, dq, dk, end;
};

BwdSpace bwd_space(const BwdPlan& p, int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk,
                   int64_t Dv) {
    BwdSpace o{};
    size_t n = 0;
    auto take = [&](size_t bytes) {
        const size_t at = n;
        n += up16(bytes);
        return at;
    };
    const size_t bh = (size_t)(B * H), state = 4 * (size_t)(Dk * Dv) * bh;
    const size_t nblk = (size_t)p.nblk, marks = (size_t)p.p.marks;
    o.s = take(state * marks);
    o.sdec = take(4 * bh * marks);
    o.g = take(state * marks);
    o.gdec = take(4 * bh * marks);
    o.sk = take(state * nblk);
    o.gk = take(state * (nblk - 1));
    const size_t dots = 4 * bh * (size_t)T * (size_t)((Dk + 15) / 16);
    o.qd = take(dots);
    o.kd = take(dots);
    o.part = take(8 * bh * nblk);
    const size_t heads = H != Hk ? 4 * bh * (size_t)T * (size_t)Dk : 0;
    o.dq = take(heads);
    o.dk = take(heads);
    o.end = n;
    return o;
}

}  // namespace

int64_t la_bwd_workgroups(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, bool bf16,
                          bool g_head) {
    const BwdPlan p = bwd_plan(B, T, H, Dk, Dv, bf16, g_head);
    const int64_t segs = p.p.nseg + p.p.marks + p.pv.nseg;
    const int64_t chain = 4 * ((B * H * segs + 7) / 8 * 8 * (2 * blocks(Dk) + blocks(Dv)));
    const int64_t states = 2 * cdiv(B * H * Dk * Dv, 256);
    const int64_t sums = B * H * p.nblk + 2 * 16384;        // the most of stride_blocks
    const int64_t most = chain > states ? chain : states;
    return most > sums ? most : sums;
}

size_t la_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                              bool bf16, bool g_head) {
    return bwd_space(bwd_plan(B, T, H, Dk, Dv, bf16, g_head), B, T, H, Hk, Dk, Dv).end;
}

hipError_t launch_la_bwd(const LaArgs& a) {
    const BwdPlan p = bwd_plan(a.B, a.T, a.H, a.Dk, a.Dv, a.bf16, a.g_head);
    const BwdSpace w = bwd_space(p, a.B, a.T, a.H, a.Hk, a.Dk, a.Dv);
    char* ws = static_cast<char*>(a.workspace);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    LaChain c = chain(a, p.p);
    c.every = p.every;

    LaJob jq = job(a.dout, a.v, a.k, a.Dv, a.Dk);
    jq.pair = jq.inter = a.scale;
    jq.h_in = a.s0;
    jq.hz = 1;
    jq.hk = a.Dk;
    LaJob jk = job(a.v, a.dout, a.q, a.Dv, a.Dk);
    jk.back = true;
    jk.pair = jk.upd = a.scale;
    jk.h_in = a.ds_final;
    jk.hz = 1;
    jk.hk = a.Dk;
    LaJob jv = job(a.k, a.q, a.dout, a.Dk, a.Dv);
    jv.back = true;
    jv.pair = jv.upd = a.scale;
    jv.h_in = a.ds_final;
    jv.hz = a.Dk;
    jv.hk = 1;

    hipError_t e;
    if (p.p.nseg > 1) {
        LaJob* const jobs[2] = {&jq, &jv};
        float* const buf[2] = {f32(w.s), f32(w.g)};
        float* const decay[2] = {f32(w.sdec), f32(w.gdec)};
        if ((e = segment_states(c, p.p, jobs, 2, buf, decay, nullptr)) != hipSuccess) return e;
        jk.h_seg = jv.h_seg;
        jk.h_step = jv.h_step;
    }
    const bool own = a.H == a.Hk;
    jq.out = own ? a.dq : f32(w.dq);
    jk.out = own ? a.dk : f32(w.dk);
    for (LaJob* j : {&jq, &jk}) {
        j->ob = a.T * a.H * a.Dk;
        j->ot = a.H * a.Dk;
        j->oh = a.Dk;
        j->out_bf16 = own && a.grad_bf16;
    }
    jv.out = a.dv;
    jv.ob = a.T * a.H * a.Dv;
    jv.ot = a.H * a.Dv;
    jv.oh = a.Dv;
    jv.out_bf16 = a.grad_bf16;
    jv.h_out = a.ds0;
    jv.end_decay = true;
    if (a.dg) {
        jq.keep = f32(w.sk);
        jq.keep_end = a.ds_final != nullptr;
        jq.r = a.q;
        jq.dots = f32(w.qd);
        jk.r = a.k;
        jk.dots = f32(w.kd);
    }
    if (a.dg || p.apart) jk.keep = f32(w.gk);
    c.njobs = p.apart ? 2 : 3;
    c.job[0] = jq;
    c.job[1] = jk;
    c.job[2] = jv;
    if ((e = launch_chain(c)) != hipSuccess) return e;
    if (p.apart) {
        jv.h_seg = jk.keep;
        jv.h_step = p.pv.L / p.every;
        c.L = p.pv.L;
        c.nseg = p.pv.nseg;
        c.njobs = 1;
        c.job[0] = jv;
        if ((e = launch_chain(c)) != hipSuccess) return e;
    }
    Share m{};
    DecayGrad d{};
    uint32_t shares = 0, decays = 0;
    if (!own) {
        m.part[0] = f32(w.dq);
        m.part[1] = f32(w.dk);
        m.out[0] = a.dq;
        m.out[1] = a.dk;
        m.bf16 = a.grad_bf16;
        m.n = a.B * a.T * a.Hk * (a.Dk / 4);
        m.share = a.H / a.Hk;
        m.D = a.Dk;
        shares = (uint32_t)stride_blocks(m.n);
    }
    if (a.dg) {
        d.B = a.B;
        d.T = a.T;
        d.H = a.H;
        d.every = p.every;
        d.nblk = p.nblk;
        d.state = c.state;
        d.nq = (int)((a.Dk + 15) / 16);
        d.q = f32(w.qd);
        d.k = f32(w.kd);
        d.skeep = f32(w.sk);
        d.gkeep = f32(w.gk);
        d.ds_final = a.ds_final;
        d.s0 = a.s0;
        d.g = a.g;
        d.g_head = a.g_head;
        d.dg = a.g_head ? nullptr : a.dg;
        d.part = a.g_head ? reinterpret_cast<double*>(ws + w.part) : nullptr;
        decays = (uint32_t)(a.B * a.H * d.nblk);
    }
    if (decays + shares == 0) return hipSuccess;
    hipLaunchKernelGGL(finish_kernel, dim3(decays + 2 * shares), dim3(256), 0, a.stream, d, m,
                       decays, shares);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.dg && a.g_head)
        hipLaunchKernelGGL(head_sum_kernel, dim3((unsigned)a.H), dim3(64), 0, a.stream, d.part,
                           a.dg, a.B * d.nblk, a.H);
    return hipGetLastError();
}

}  // namespace gdr
