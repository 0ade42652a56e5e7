// C ABI of linear attention, rotary positions and RMS norm (declared in
// gdr_linear.h).  Host-side validation and dispatch; an error status means nothing
// was launched.
#include <algorithm>
#include <array>
#include <cmath>
#include <initializer_list>

#include "../../include/gdr_linear.h"
#include "api_checks.h"
#include "block_launch.h"
#include "linear_launch.h"

using namespace gdr;

namespace {

size_t elem(gdr_dtype_t d) { return d == GDR_BF16 ? 2 : 4; }

bool opt_elem(const void* p, size_t bytes) { return !p || elem_ok(p, bytes); }

using Ptrs = std::initializer_list<const void*>;

// Whether none of the outputs starts at an input or at another output (NULL ones
// aside).
bool apart(Ptrs outs, Ptrs ins) {
    for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
        if (!*o) continue;
        for (const void* p : ins)
            if (p == *o) return false;
        for (const void* const* q = outs.begin(); q != o; ++q)
            if (*q == *o) return false;
    }
    return true;
}

bool strides_ok(const int64_t* s, int n) {
    for (int i = 0; s && i < n; ++i)
        if (s[i] < 0 || s[i] > ((int64_t)1 << 40)) return false;
    return true;
}

// Whether the rows of `d` elements at every multiple of the strides lie apart: by
// growing stride, each passes what the dimensions before it take up.
bool places_apart(std::array<int64_t, 3> n, std::array<int64_t, 3> stride, int64_t d) {
    std::array<int, 3> order{0, 1, 2};
    std::sort(order.begin(), order.end(), [&](int i, int j) { return stride[i] < stride[j]; });
    double span = (double)d;
    for (int i : order) {
        if (n[i] <= 1) continue;
        if ((double)stride[i] < span) return false;
        span += (double)stride[i] * (double)(n[i] - 1);
    }
    return true;
}

bool workgroups_ok(double n) { return n * 256.0 <= (double)kMaxWorkItems; }

// Sizes whose products stay below 2^62, so that they can be formed.
bool product_ok(std::initializer_list<int64_t> v) {
    double n = 1.0;
    for (int64_t x : v) {
        if (x < 0) return false;
        n *= (double)(x > 0 ? x : 1);
    }
    return n < 4.0e18;
}

__global__ __launch_bounds__(256) void fill_kernel(const float* __restrict__ s,
                                                   float* __restrict__ d, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        d[i] = s ? s[i] : 0.f;
}

// d = s, or zeros.
gdr_status_t copy_or_zero(const float* s, float* d, int64_t n, hipStream_t st) {
    if (n == 0 || s == d) return GDR_OK;
    hipLaunchKernelGGL(fill_kernel, dim3(stride_blocks(n)), dim3(256), 0, st, s, d, n);
    return from_hip(hipGetLastError());
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t* __restrict__ d, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        d[i] = 0;
}

// n elements at any element's alignment.
gdr_status_t zero_elements(void* d, gdr_dtype_t dt, int64_t n, hipStream_t st) {
    const int64_t words = n * (int64_t)(elem(dt) / 2);
    hipLaunchKernelGGL(zero_kernel, dim3(stride_blocks(words)), dim3(256), 0, st,
                       static_cast<uint16_t*>(d), words);
    return from_hip(hipGetLastError());
}

// Tensor i of [B, T, heads, d] with the caller's strides or contiguous.
LaTensor tensor(const void* p, const int64_t* s, int i, int64_t T, int64_t heads, int64_t d,
                int64_t share) {
    LaTensor t{};
    t.p = p;
    t.sb = s ? s[3 * i] : T * heads * d;
    t.st = s ? s[3 * i + 1] : heads * d;
    t.sh = s ? s[3 * i + 2] : d;
    t.share = share;
    return t;
}

gdr_status_t la_check(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                      gdr_dtype_t in_dt, gdr_dtype_t other_dt, uint32_t flags) {
    if (B < 0 || T < 0 || H < 0 || Hk < 0 || Dk < 0 || Dv < 0) return GDR_ERR_INVALID;
    if (!dtype_ok(in_dt) || !dtype_ok(other_dt) || (flags & ~GDR_LA_HEAD_DECAY))
        return GDR_ERR_UNSUPPORTED;
    if (Dk < 8 || Dv < 8 || Dk % 8 || Dv % 8 || Dk > GDR_LA_MAX_D || Dv > GDR_LA_MAX_D)
        return GDR_ERR_UNSUPPORTED;
    if (H > GDR_MAX_HEADS || (H > 0 && (Hk == 0 || H % Hk))) return GDR_ERR_INVALID;
    // room for every product of sizes that the launchers form
    if (T > ((int64_t)1 << 40) || !product_ok({B, T + 1024, H, 1 << 16})) return GDR_ERR_INVALID;
    return GDR_OK;
}

// Token strides: 64 tokens of a chunk lie within 32-bit byte offsets.
bool token_strides_ok(const int64_t* s, int n) {
    for (int i = 0; s && i < n; ++i)
        if (s[3 * i + 1] > GDR_LA_MAX_TOKEN_STRIDE) return false;
    return true;
}

bool la_nothing(int64_t B, int64_t H) { return B == 0 || H == 0; }

}  // namespace

extern "C" size_t gdr_linear_attn_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t Dk,
                                                     int64_t Dv, gdr_dtype_t in_dt) {
    if (la_check(B, T, H, H, Dk, Dv, in_dt, in_dt, 0) != GDR_OK || la_nothing(B, H) || T == 0 ||
        !workgroups_ok((double)la_fwd_workgroups(B, T, H, Dk, Dv, in_dt == GDR_BF16)))
        return 0;
    return la_fwd_workspace_bytes(B, T, H, Dk, Dv, in_dt == GDR_BF16);
}

extern "C" gdr_status_t gdr_linear_attn_fwd(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk,
                                            int64_t Dv, gdr_dtype_t in_dt, const void* q,
                                            const void* k, const void* v, const int64_t* strides,
                                            const float* log_decay, const float* s0, float scale,
                                            uint32_t flags, gdr_dtype_t out_dt, void* o,
                                            float* s_final, void* workspace,
                                            size_t workspace_bytes, hipStream_t stream) {
    const gdr_status_t st = la_check(B, T, H, Hk, Dk, Dv, in_dt, out_dt, flags);
    if (st != GDR_OK) return st;
    if (!strides_ok(strides, 9) || !token_strides_ok(strides, 3)) return GDR_ERR_INVALID;
    if (la_nothing(B, H)) return GDR_OK;
    if (!opt_elem(s0, 4) || !opt_elem(s_final, 4)) return GDR_ERR_INVALID;
    if (T == 0) return s_final ? copy_or_zero(s0, s_final, B * H * Dk * Dv, stream) : GDR_OK;
    const size_t ie = elem(in_dt);
    if (!elem_ok(q, ie) || !elem_ok(k, ie) || !elem_ok(v, ie) || !opt_elem(log_decay, 4) ||
        !elem_ok(o, elem(out_dt)))
        return GDR_ERR_INVALID;
    const bool bf = in_dt == GDR_BF16;
    if (!workgroups_ok((double)la_fwd_workgroups(B, T, H, Dk, Dv, bf))) return GDR_ERR_INVALID;
    const size_t need = la_fwd_workspace_bytes(B, T, H, Dk, Dv, bf);
    if (need && (!ptrs_ok({workspace}) || workspace_bytes < need)) return GDR_ERR_INVALID;
    if (!apart({o, s_final, need ? workspace : nullptr}, {q, k, v, log_decay}) ||
        !apart({o, need ? workspace : nullptr}, {s0}))
        return GDR_ERR_INVALID;
    LaArgs a{};
    a.B = B;
    a.T = T;
    a.H = H;
    a.Hk = Hk;
    a.Dk = Dk;
    a.Dv = Dv;
    a.bf16 = bf;
    a.q = tensor(q, strides, 0, T, Hk, Dk, H / Hk);
    a.k = tensor(k, strides, 1, T, Hk, Dk, H / Hk);
    a.v = tensor(v, strides, 2, T, H, Dv, 1);
    a.g = log_decay;
    a.g_head = flags & GDR_LA_HEAD_DECAY;
    a.s0 = s0;
    a.scale = scale;
    a.out_bf16 = out_dt == GDR_BF16;
    a.o = o;
    a.s_final = s_final;
    a.workspace = workspace;
    a.stream = stream;
    return from_hip(launch_la_fwd(a));
}

extern "C" gdr_status_t gdr_linear_attn_step(int64_t N, int64_t H, int64_t Hk, int64_t Dk,
                                             int64_t Dv, gdr_dtype_t in_dt, const void* q,
                                             const void* k, const void* v, const int64_t* strides,
                                             const float* log_decay, float* state, float scale,
                                             uint32_t flags, gdr_dtype_t out_dt, void* o,
                                             hipStream_t stream) {
    const gdr_status_t st = la_check(N, 1, H, Hk, Dk, Dv, in_dt, out_dt, flags);
    if (st != GDR_OK) return st;
    if (!strides_ok(strides, 6)) return GDR_ERR_INVALID;
    if (la_nothing(N, H)) return GDR_OK;
    const size_t ie = elem(in_dt);
    if (!elem_ok(q, ie) || !elem_ok(k, ie) || !elem_ok(v, ie) || !opt_elem(log_decay, 4) ||
        !elem_ok(state, 4) || !elem_ok(o, elem(out_dt)))
        return GDR_ERR_INVALID;
    if (!apart({o, state}, {q, k, v, log_decay})) return GDR_ERR_INVALID;
    if (!workgroups_ok((double)la_step_workgroups(N, H, Dk, Dv))) return GDR_ERR_INVALID;
    int64_t s[9];
    for (int i = 0; strides && i < 3; ++i) {
        s[3 * i] = strides[2 * i];
        s[3 * i + 1] = 0;
        s[3 * i + 2] = strides[2 * i + 1];
    }
    const int64_t* sp = strides ? s : nullptr;
    LaStepArgs a{};
    a.N = N;
    a.H = H;
    a.Hk = Hk;
    a.Dk = Dk;
    a.Dv = Dv;
    a.bf16 = in_dt == GDR_BF16;
    a.out_bf16 = out_dt == GDR_BF16;
    a.q = tensor(q, sp, 0, 1, Hk, Dk, H / Hk);
    a.k = tensor(k, sp, 1, 1, Hk, Dk, H / Hk);
    a.v = tensor(v, sp, 2, 1, H, Dv, 1);
    a.g = log_decay;
    a.g_head = flags & GDR_LA_HEAD_DECAY;
    a.scale = scale;
    a.state = state;
    a.o = o;
    a.stream = stream;
    return from_hip(launch_la_step(a));
}

extern "C" size_t gdr_linear_attn_bwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t Hk,
                                                     int64_t Dk, int64_t Dv, gdr_dtype_t in_dt,
                                                     uint32_t flags) {
    const bool bf = in_dt == GDR_BF16, head = flags & GDR_LA_HEAD_DECAY;
    if (la_check(B, T, H, Hk, Dk, Dv, in_dt, in_dt, flags) != GDR_OK || la_nothing(B, H) ||
        T == 0 || !workgroups_ok((double)la_bwd_workgroups(B, T, H, Dk, Dv, bf, head)))
        return 0;
    return la_bwd_workspace_bytes(B, T, H, Hk, Dk, Dv, bf, head);
}

extern "C" gdr_status_t gdr_linear_attn_bwd(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk,
                                            int64_t Dv, gdr_dtype_t in_dt, const void* q,
                                            const void* k, const void* v, const int64_t* strides,
                                            const float* log_decay, const float* s0,
                                            const void* dout, const float* ds_final, float scale,
                                            uint32_t flags, gdr_dtype_t grad_dt, void* dq,
                                            void* dk, void* dv, float* dlog_decay, float* ds0,
                                            void* workspace, size_t workspace_bytes,
                                            hipStream_t stream) {
    const gdr_status_t st = la_check(B, T, H, Hk, Dk, Dv, in_dt, grad_dt, flags);
    if (st != GDR_OK) return st;
    if (!strides_ok(strides, 12) || !token_strides_ok(strides, 4)) return GDR_ERR_INVALID;
    if (H == 0) {
        // heads of q and k that no head of v reads: the sums over none
        if (B == 0 || T == 0 || Hk == 0) return GDR_OK;
        if (!product_ok({B, T, Hk, Dk}) || !elem_ok(dq, elem(grad_dt)) ||
            !elem_ok(dk, elem(grad_dt)) || !apart({dq, dk}, {q, k}))
            return GDR_ERR_INVALID;
        const gdr_status_t e = zero_elements(dq, grad_dt, B * T * Hk * Dk, stream);
        return e == GDR_OK ? zero_elements(dk, grad_dt, B * T * Hk * Dk, stream) : e;
    }
    if (!opt_elem(s0, 4) || !opt_elem(ds_final, 4) || !opt_elem(ds0, 4) ||
        !opt_elem(dlog_decay, 4) || !opt_elem(log_decay, 4) || (dlog_decay && T && B && !log_decay))
        return GDR_ERR_INVALID;
    const bool head = flags & GDR_LA_HEAD_DECAY;
    if (B == 0 || T == 0) {
        gdr_status_t e = GDR_OK;
        if (dlog_decay && head) e = copy_or_zero(nullptr, dlog_decay, H, stream);
        if (e == GDR_OK && ds0 && B > 0)
            e = copy_or_zero(ds_final, ds0, B * H * Dk * Dv, stream);
        return e;
    }
    const size_t ie = elem(in_dt), ge = elem(grad_dt);
    if (!elem_ok(q, ie) || !elem_ok(k, ie) || !elem_ok(v, ie) || !elem_ok(dout, ie) ||
        !elem_ok(dq, ge) || !elem_ok(dk, ge) || !elem_ok(dv, ge))
        return GDR_ERR_INVALID;
    if (!apart({dq, dk, dv, dlog_decay, ds0, workspace}, {q, k, v, log_decay, s0, dout, ds_final}))
        return GDR_ERR_INVALID;
    const bool bf = in_dt == GDR_BF16;
    if (!workgroups_ok((double)la_bwd_workgroups(B, T, H, Dk, Dv, bf, head)))
        return GDR_ERR_INVALID;
    if (!ptrs_ok({workspace}) ||
        workspace_bytes < la_bwd_workspace_bytes(B, T, H, Hk, Dk, Dv, bf, head))
        return GDR_ERR_INVALID;
    LaArgs a{};
    a.B = B;
    a.T = T;
    a.H = H;
    a.Hk = Hk;
    a.Dk = Dk;
    a.Dv = Dv;
    a.bf16 = bf;
    a.q = tensor(q, strides, 0, T, Hk, Dk, H / Hk);
    a.k = tensor(k, strides, 1, T, Hk, Dk, H / Hk);
    a.v = tensor(v, strides, 2, T, H, Dv, 1);
    a.dout = tensor(dout, strides, 3, T, H, Dv, 1);
    a.g = log_decay;
    a.g_head = head;
    a.s0 = s0;
    a.scale = scale;
    a.ds_final = ds_final;
    a.grad_bf16 = grad_dt == GDR_BF16;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dg = dlog_decay;
    a.ds0 = ds0;
    a.workspace = workspace;
    a.stream = stream;
    return from_hip(launch_la_bwd(a));
}

extern "C" gdr_status_t gdr_rotary(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                                   int64_t rot, gdr_dtype_t dt, const void* q, const void* k,
                                   const int64_t* strides, const int64_t* positions,
                                   int64_t pos_stride, int64_t start, const double* freqs,
                                   float scale, uint32_t flags, void* q_out, void* k_out,
                                   hipStream_t stream) {
    if (B < 0 || T < 0 || Hq < 0 || Hk < 0 || D < 0) return GDR_ERR_INVALID;
    if (!dtype_ok(dt) || (flags & ~(GDR_ROTARY_INTERLEAVED | GDR_ROTARY_INVERSE)) ||
        D > GDR_ROTARY_MAX_D)
        return GDR_ERR_UNSUPPORTED;
    if (rot <= 0 || rot % 2 || rot > D) return GDR_ERR_INVALID;
    if (Hq > GDR_MAX_HEADS || Hk > GDR_MAX_HEADS - Hq || !strides_ok(strides, 12) ||
        !strides_ok(&pos_stride, 1) || !product_ok({B, T, Hq + Hk, D}))
        return GDR_ERR_INVALID;
    if (B == 0 || T == 0 || Hq + Hk == 0) return GDR_OK;
    // the last position is a 64-bit number too
    if (!positions && start > INT64_MAX - (T - 1)) return GDR_ERR_INVALID;
    const size_t e = elem(dt);
    if ((Hq && (!elem_ok(q, e) || !elem_ok(q_out, e))) ||
        (Hk && (!elem_ok(k, e) || !elem_ok(k_out, e))) || !opt_elem(positions, 8) ||
        !elem_ok(freqs, 8))
        return GDR_ERR_INVALID;
    if (!Hq) q = q_out = nullptr;
    if (!Hk) k = k_out = nullptr;
    RotaryArgs a{};
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.Hk = Hk;
    a.D = D;
    a.rot = rot;
    a.bf16 = dt == GDR_BF16;
    a.interleaved = flags & GDR_ROTARY_INTERLEAVED;
    a.inverse = flags & GDR_ROTARY_INVERSE;
    const LaTensor qi = tensor(q, strides, 0, T, Hq, D, 1), ki = tensor(k, strides, 1, T, Hk, D, 1);
    const LaTensor qo = tensor(q_out, strides, 2, T, Hq, D, 1);
    const LaTensor ko = tensor(k_out, strides, 3, T, Hk, D, 1);
    a.q = {q, q_out, qi.sb, qi.st, qi.sh, qo.sb, qo.st, qo.sh};
    a.k = {k, k_out, ki.sb, ki.st, ki.sh, ko.sb, ko.st, ko.sh};
    for (const RotarySide* s : {&a.q, &a.k}) {
        if (!s->out) continue;
        const int64_t heads = s == &a.q ? Hq : Hk;
        if (!places_apart({B, T, heads}, {s->ob, s->ot, s->oh}, D)) return GDR_ERR_INVALID;
        // in place: every element where it was
        if (s->in == s->out && ((B > 1 && s->ib != s->ob) || (T > 1 && s->it != s->ot) ||
                                (heads > 1 && s->ih != s->oh)))
            return GDR_ERR_INVALID;
    }
    if (!apart({q_out, k_out}, {positions, freqs}) || !apart({q_out}, {k}) || !apart({k_out}, {q}))
        return GDR_ERR_INVALID;
    a.positions = positions;
    a.pos_stride = pos_stride;
    a.start = start;
    a.freqs = freqs;
    a.scale = scale;
    a.stream = stream;
    rotary_shape(a);
    if (rotary_work_items(a) > (double)kMaxWorkItems) return GDR_ERR_INVALID;
    return from_hip(launch_rotary(a));
}

extern "C" gdr_status_t gdr_rotary_frequencies(int64_t rot, double base,
                                               gdr_rotary_scaling_t scaling, double factor,
                                               double low, double high, double original,
                                               double* freqs) {
    if (rot <= 0 || rot % 2 || rot > GDR_ROTARY_MAX_D || !freqs) return GDR_ERR_INVALID;
    if (!(base > 0.0) || !std::isfinite(base)) return GDR_ERR_INVALID;
    if (scaling < GDR_ROTARY_PLAIN || scaling > GDR_ROTARY_PARTS) return GDR_ERR_UNSUPPORTED;
    if (scaling != GDR_ROTARY_PLAIN && !(factor > 0.0 && std::isfinite(factor)))
        return GDR_ERR_INVALID;
    if (scaling == GDR_ROTARY_BASE) {
        if (rot == 2) return GDR_ERR_INVALID;
        base *= std::pow(factor, (double)rot / (double)(rot - 2));
    }
    if (scaling == GDR_ROTARY_PARTS &&
        !(low >= 0.0 && high > low && std::isfinite(high) && original > 0.0 &&
          std::isfinite(original)))
        return GDR_ERR_INVALID;
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * (double)i / (double)rot);
        if (scaling == GDR_ROTARY_LINEAR) f /= factor;
        if (scaling == GDR_ROTARY_PARTS) {
            const double turns = original * f / 6.283185307179586;
            double w = (turns - low) / (high - low);
            w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
            f *= w + (1.0 - w) / factor;
        }
        freqs[i] = f;
    }
    return GDR_OK;
}

static gdr_status_t rms_check(int64_t R, int64_t C, gdr_dtype_t a, gdr_dtype_t b, gdr_dtype_t c,
                              float eps) {
    if (R < 0 || C < 0) return GDR_ERR_INVALID;
    if (!dtype_ok(a) || !dtype_ok(b) || !dtype_ok(c) || C > GDR_RMS_MAX_C)
        return GDR_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return GDR_ERR_INVALID;
    if (!product_ok({R, C, 16})) return GDR_ERR_INVALID;
    return GDR_OK;
}

// What both forwards check; fills everything but the output.
static gdr_status_t rms_fill(RmsArgs& a, int64_t R, int64_t C, gdr_dtype_t in_dt, const void* x,
                             int64_t x_stride, gdr_dtype_t res_dt, const void* res,
                             int64_t res_stride, const float* w, float eps, void* h) {
    if (!elem_ok(x, elem(in_dt)) || !opt_elem(w, 4)) return GDR_ERR_INVALID;
    if ((res != nullptr) != (h != nullptr)) return GDR_ERR_INVALID;
    if (!opt_elem(res, elem(res_dt)) || !opt_elem(h, elem(res_dt))) return GDR_ERR_INVALID;
    if (h && h == res && res_stride != C && R > 1) return GDR_ERR_INVALID;
    if (!apart({h}, {x, w})) return GDR_ERR_INVALID;
    if (rms_work_items(R, C) > (double)kMaxWorkItems) return GDR_ERR_INVALID;
    a.R = R;
    a.C = C;
    a.in_bf16 = in_dt == GDR_BF16;
    a.res_bf16 = res_dt == GDR_BF16;
    a.x = x;
    a.xr = x_stride;
    a.res = res;
    a.rr = res_stride;
    a.w = w;
    a.eps = eps;
    a.h = h;
    return GDR_OK;
}

extern "C" gdr_status_t gdr_rms_norm_fwd(int64_t R, int64_t C, gdr_dtype_t in_dt, const void* x,
                                         int64_t x_stride, gdr_dtype_t res_dt, const void* res,
                                         int64_t res_stride, const float* w, float eps,
                                         gdr_dtype_t out_dt, void* y, void* h,
                                         hipStream_t stream) {
    gdr_status_t st = rms_check(R, C, in_dt, res_dt, out_dt, eps);
    if (st != GDR_OK) return st;
    if (!strides_ok(&x_stride, 1) || !strides_ok(&res_stride, 1)) return GDR_ERR_INVALID;
    if (R == 0 || C == 0) return GDR_OK;
    RmsArgs a{};
    st = rms_fill(a, R, C, in_dt, x, x_stride, res_dt, res, res_stride, w, eps, h);
    if (st != GDR_OK) return st;
    if (!elem_ok(y, elem(out_dt)) || !apart({y, h}, {w}) || !apart({y}, {res}))
        return GDR_ERR_INVALID;
    if (y == x && (in_dt != out_dt || (x_stride != C && R > 1))) return GDR_ERR_INVALID;
    a.out_bf16 = out_dt == GDR_BF16;
    a.y = y;
    a.stream = stream;
    return from_hip(launch_rms_fwd(a));
}

extern "C" gdr_status_t gdr_rms_norm_quant(int64_t R, int64_t C, gdr_dtype_t in_dt, const void* x,
                                           int64_t x_stride, gdr_dtype_t res_dt, const void* res,
                                           int64_t res_stride, const float* w, float eps,
                                           gdr_q8_t type, int64_t group, void* y, float* scales,
                                           void* h, hipStream_t stream) {
    gdr_status_t st = rms_check(R, C, in_dt, res_dt, in_dt, eps);
    if (st != GDR_OK) return st;
    if (type != GDR_Q_E4M3 && type != GDR_Q_INT8) return GDR_ERR_UNSUPPORTED;
    if (group != 0 && group != 32 && group != 64 && group != 128) return GDR_ERR_UNSUPPORTED;
    if (group && C % group) return GDR_ERR_INVALID;
    if (!strides_ok(&x_stride, 1) || !strides_ok(&res_stride, 1)) return GDR_ERR_INVALID;
    if (R == 0 || C == 0) return GDR_OK;
    RmsArgs a{};
    st = rms_fill(a, R, C, in_dt, x, x_stride, res_dt, res, res_stride, w, eps, h);
    if (st != GDR_OK) return st;
    if (!y || !elem_ok(scales, 4) || !apart({y, scales, h}, {x, w}) || !apart({y, scales}, {res}))
        return GDR_ERR_INVALID;
    a.q8 = type == GDR_Q_E4M3 ? 1 : 2;
    a.group = group ? group : C;
    a.y = y;
    a.scales = scales;
    a.stream = stream;
    return from_hip(launch_rms_fwd(a));
}

// The second launch of the backward: up to 1024 threads for 64 columns.
static bool rms_bwd_ok(int64_t R, int64_t C) {
    return rms_work_items(R, C) <= (double)kMaxWorkItems && workgroups_ok((double)C / 16.0);
}

extern "C" size_t gdr_rms_norm_bwd_workspace_size(int64_t R, int64_t C) {
    if (R <= 0 || C <= 0 || rms_check(R, C, GDR_F32, GDR_F32, GDR_F32, 0.f) != GDR_OK ||
        !rms_bwd_ok(R, C))
        return 0;
    return rms_bwd_workspace_bytes(R, C);
}

extern "C" gdr_status_t gdr_rms_norm_bwd(int64_t R, int64_t C, gdr_dtype_t in_dt, const void* x,
                                         int64_t x_stride, const float* w, gdr_dtype_t dy_dt,
                                         const void* dy, int64_t dy_stride, float eps,
                                         gdr_dtype_t grad_dt, const void* dres,
                                         int64_t dres_stride, void* dx, float* dw,
                                         void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
    const gdr_status_t st = rms_check(R, C, in_dt, dy_dt, grad_dt, eps);
    if (st != GDR_OK) return st;
    if (!strides_ok(&x_stride, 1) || !strides_ok(&dy_stride, 1) || !strides_ok(&dres_stride, 1))
        return GDR_ERR_INVALID;
    if (C == 0) return GDR_OK;
    if (!opt_elem(dw, 4)) return GDR_ERR_INVALID;
    if (R == 0) return dw ? copy_or_zero(nullptr, dw, C, stream) : GDR_OK;
    const size_t ge = elem(grad_dt);
    if (!elem_ok(x, elem(in_dt)) || !opt_elem(w, 4) || !elem_ok(dy, elem(dy_dt)) ||
        !elem_ok(dx, ge) || !opt_elem(dres, ge))
        return GDR_ERR_INVALID;
    if (!apart({dx, dw, dw ? workspace : nullptr}, {x, w, dy}) ||
        !apart({dw, dw ? workspace : nullptr}, {dres}))
        return GDR_ERR_INVALID;
    if (dx == dres && dres_stride != C && R > 1) return GDR_ERR_INVALID;
    if (!rms_bwd_ok(R, C)) return GDR_ERR_INVALID;
    if (dw && (!ptrs_ok({workspace}) || workspace_bytes < rms_bwd_workspace_bytes(R, C)))
        return GDR_ERR_INVALID;
    RmsBwdArgs a{};
    a.R = R;
    a.C = C;
    a.in_bf16 = in_dt == GDR_BF16;
    a.dy_bf16 = dy_dt == GDR_BF16;
    a.grad_bf16 = grad_dt == GDR_BF16;
    a.x = x;
    a.xr = x_stride;
    a.dy = dy;
    a.yr = dy_stride;
    a.dres = dres;
    a.rr = dres_stride;
    a.w = w;
    a.eps = eps;
    a.dx = dx;
    a.dw = dw;
    a.part = dw ? static_cast<float*>(workspace) : nullptr;
    a.stream = stream;
    return from_hip(launch_rms_bwd(a));
}
