// C ABI of the operators around the token mixer (declared in gdr_block.h): short
// causal convolution, selective state space scan, layer norm.  Host-side
// validation and dispatch; an error status means nothing was launched.
#include <initializer_list>

#include "../../include/gdr_block.h"
#include "api_checks.h"
#include "block_launch.h"

using namespace gdr;

namespace {

size_t elem(gdr_dtype_t d) { return d == GDR_BF16 ? 2 : 4; }

// NULL, or aligned to its element.
bool opt_elem(const void* p, size_t bytes) { return !p || elem_ok(p, bytes); }

using Ptrs = std::initializer_list<const void*>;

// Whether none of the outputs starts at an input or at another output (NULL ones
// aside): what a call cannot do in place it refuses.
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

// Products of sizes stay far below 2^63, strides below 2^40 elements.
bool strides_ok(const int64_t* s, int n) {
    for (int i = 0; s && i < n; ++i)
        if (s[i] < 0 || s[i] > ((int64_t)1 << 40)) return false;
    return true;
}

bool workgroups_ok(double n) { return n * 256.0 <= (double)kMaxWorkItems; }

// Strides (sequence, token) of tensor i, or those of a contiguous [B, T, C].
void pick(const int64_t* s, int i, int64_t T, int64_t C, int64_t& sb, int64_t& st) {
    sb = s ? s[2 * i] : T * C;
    st = s ? s[2 * i + 1] : C;
}

bool conv_sizes_ok(int64_t B, int64_t T, int64_t C) {
    return sizes_ok(B, T, C) && B <= ((int64_t)1 << 31) && T <= ((int64_t)1 << 40) &&
           C <= ((int64_t)1 << 31);
}

gdr_status_t conv_check(int64_t B, int64_t T, int64_t C, int64_t K, gdr_dtype_t in_dt,
                        gdr_dtype_t other_dt, uint32_t flags) {
    if (B < 0 || T < 0 || C < 0) return GDR_ERR_INVALID;
    if (!conv_sizes_ok(B, T, C) || !sizes_ok(B, T + 8, C)) return GDR_ERR_INVALID;
    if (!dtype_ok(in_dt) || !dtype_ok(other_dt)) return GDR_ERR_UNSUPPORTED;
    if (K < 2 || K > 4 || (flags & ~GDR_CONV_SILU)) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

__global__ __launch_bounds__(256) void copy_words(const uint16_t* __restrict__ s,
                                                  uint16_t* __restrict__ d, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        d[i] = s ? s[i] : (uint16_t)0;
}

// d = s, or zeros; n bytes, even (states of any dtype).
gdr_status_t copy_or_zero(const void* s, void* d, int64_t bytes, hipStream_t st) {
    if (bytes == 0 || s == d) return GDR_OK;
    hipLaunchKernelGGL(copy_words, dim3(stride_blocks(bytes / 2)), dim3(256), 0, st,
                       (const uint16_t*)s, (uint16_t*)d, bytes / 2);
    return from_hip(hipGetLastError());
}

}  // namespace

extern "C" gdr_status_t gdr_short_conv_fwd(int64_t B, int64_t T, int64_t C, int64_t K,
                                           gdr_dtype_t in_dt, const void* x,
                                           const int64_t* strides, const float* w,
                                           const float* bias, const void* s0, uint32_t flags,
                                           gdr_dtype_t out_dt, void* y, void* s_final,
                                           hipStream_t stream) {
    const gdr_status_t st = conv_check(B, T, C, K, in_dt, out_dt, flags);
    if (st != GDR_OK) return st;
    if (!strides_ok(strides, 2)) return GDR_ERR_INVALID;
    if (B == 0 || C == 0) return GDR_OK;
    const size_t ie = elem(in_dt);
    if (!opt_elem(s0, ie) || !opt_elem(s_final, ie)) return GDR_ERR_INVALID;
    if (T == 0)
        return s_final ? copy_or_zero(s0, s_final, B * (K - 1) * C * (int64_t)ie, stream) : GDR_OK;
    if (!elem_ok(x, ie) || !elem_ok(y, elem(out_dt)) || !elem_ok(w, 4) || !opt_elem(bias, 4))
        return GDR_ERR_INVALID;
    if (!apart({y, s_final}, {x, w, bias}) || !apart({y}, {s0})) return GDR_ERR_INVALID;
    if (!workgroups_ok((double)conv_workgroups(B, T, C))) return GDR_ERR_INVALID;
    ConvArgs a{};
    a.B = B;
    a.T = T;
    a.C = C;
    a.K = (int)K;
    a.in_bf16 = in_dt == GDR_BF16;
    a.out_bf16 = out_dt == GDR_BF16;
    a.silu = flags & GDR_CONV_SILU;
    a.x = x;
    pick(strides, 0, T, C, a.xb, a.xt);
    a.w = w;
    a.bias = bias;
    a.s0 = s0;
    a.y = y;
    a.s_final = s_final;
    a.stream = stream;
    return from_hip(launch_conv_fwd(a));
}

extern "C" gdr_status_t gdr_short_conv_step(int64_t N, int64_t C, int64_t K, gdr_dtype_t in_dt,
                                            const void* x, int64_t x_stride, const float* w,
                                            const float* bias, void* state, uint32_t flags,
                                            gdr_dtype_t out_dt, void* y, hipStream_t stream) {
    const gdr_status_t st = conv_check(N, 1, C, K, in_dt, out_dt, flags);
    if (st != GDR_OK) return st;
    if (!strides_ok(&x_stride, 1)) return GDR_ERR_INVALID;
    if (N == 0 || C == 0) return GDR_OK;
    if (!elem_ok(x, elem(in_dt)) || !elem_ok(state, elem(in_dt)) || !elem_ok(y, elem(out_dt)) ||
        !elem_ok(w, 4) || !opt_elem(bias, 4))
        return GDR_ERR_INVALID;
    if (!apart({y, state}, {x, w, bias})) return GDR_ERR_INVALID;
    if (!workgroups_ok((double)N * (double)((C + 3) / 4) / 256.0 + 1.0)) return GDR_ERR_INVALID;
    ConvArgs a{};
    a.B = N;
    a.T = 1;
    a.C = C;
    a.K = (int)K;
    a.in_bf16 = in_dt == GDR_BF16;
    a.out_bf16 = out_dt == GDR_BF16;
    a.silu = flags & GDR_CONV_SILU;
    a.x = x;
    a.xb = x_stride;
    a.w = w;
    a.bias = bias;
    a.s0 = state;
    a.s_final = state;
    a.y = y;
    a.stream = stream;
    return from_hip(launch_conv_step(a));
}

// The second launch of the convolution's backward: up to 1024 threads for 64
// columns.
static bool conv_sums_ok(int64_t C, int64_t K) {
    return workgroups_ok((double)C * (double)(K + 1) / 16.0);
}

extern "C" size_t gdr_short_conv_bwd_workspace_size(int64_t B, int64_t T, int64_t C, int64_t K) {
    if (B <= 0 || T <= 0 || C <= 0 ||
        conv_check(B, T, C, K, GDR_F32, GDR_F32, 0) != GDR_OK || !conv_sums_ok(C, K))
        return 0;
    return conv_bwd_workspace_bytes(B, T, C, K);
}

extern "C" gdr_status_t gdr_short_conv_bwd(int64_t B, int64_t T, int64_t C, int64_t K,
                                           gdr_dtype_t in_dt, const void* x, const float* w,
                                           const float* bias, const void* s0, gdr_dtype_t dy_dt,
                                           const void* dy, const int64_t* strides,
                                           const float* ds_final, uint32_t flags,
                                           gdr_dtype_t grad_dt, void* dx, float* dw, float* dbias,
                                           float* ds0, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
    const gdr_status_t st = conv_check(B, T, C, K, in_dt, dy_dt, flags);
    if (st != GDR_OK) return st;
    if (!dtype_ok(grad_dt)) return GDR_ERR_UNSUPPORTED;
    if (!strides_ok(strides, 4)) return GDR_ERR_INVALID;
    if (C == 0) return GDR_OK;
    if (!opt_elem(dw, 4) || !opt_elem(dbias, 4) || !opt_elem(ds0, 4) || !opt_elem(ds_final, 4))
        return GDR_ERR_INVALID;
    if (B == 0 || T == 0) {
        gdr_status_t e = GDR_OK;
        if (dw) e = copy_or_zero(nullptr, dw, C * K * 4, stream);
        if (e == GDR_OK && dbias) e = copy_or_zero(nullptr, dbias, C * 4, stream);
        if (e == GDR_OK && ds0 && B > 0)
            e = copy_or_zero(ds_final, ds0, B * (K - 1) * C * 4, stream);
        return e;
    }
    const size_t ie = elem(in_dt);
    if (!elem_ok(x, ie) || !elem_ok(w, 4) || !opt_elem(bias, 4) || !opt_elem(s0, ie) ||
        !elem_ok(dy, elem(dy_dt)) || !elem_ok(dx, elem(grad_dt)))
        return GDR_ERR_INVALID;
    const bool sums = dw || dbias;
    if (!apart({dx, dw, dbias, ds0, sums ? workspace : nullptr}, {x, w, bias, s0, dy, ds_final}))
        return GDR_ERR_INVALID;
    if (sums && (!ptrs_ok({workspace}) ||
                 workspace_bytes < conv_bwd_workspace_bytes(B, T, C, K)))
        return GDR_ERR_INVALID;
    if (sums && !conv_sums_ok(C, K)) return GDR_ERR_INVALID;
    ConvArgs a{};
    a.B = B;
    a.T = T;
    a.C = C;
    a.K = (int)K;
    a.in_bf16 = in_dt == GDR_BF16;
    a.dy_bf16 = dy_dt == GDR_BF16;
    a.grad_bf16 = grad_dt == GDR_BF16;
    a.silu = flags & GDR_CONV_SILU;
    a.x = x;
    pick(strides, 0, T, C, a.xb, a.xt);
    a.w = w;
    a.bias = bias;
    a.s0 = s0;
    a.dy = dy;
    pick(strides, 1, T, C, a.yb, a.yt);
    a.ds_final = ds_final;
    a.dx = dx;
    a.dw = dw;
    a.dbias = dbias;
    a.ds0 = ds0;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.stream = stream;
    return from_hip(launch_conv_bwd(a));
}

static gdr_status_t norm_check(int64_t R, int64_t C, gdr_dtype_t a, gdr_dtype_t b, gdr_dtype_t c,
                               float eps) {
    if (R < 0 || C < 0 || !sizes_ok(R, C, 1)) return GDR_ERR_INVALID;
    if (!dtype_ok(a) || !dtype_ok(b) || !dtype_ok(c)) return GDR_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || eps > 3.0e38f) return GDR_ERR_INVALID;
    if (C > GDR_NORM_MAX_C) return GDR_ERR_UNSUPPORTED;
    if (!workgroups_ok((double)R)) return GDR_ERR_INVALID;
    return GDR_OK;
}

// Whether rows `stride` apart lie as the contiguous output's do (one row always).
static bool packed(int64_t R, int64_t C, int64_t stride) { return R == 1 || stride == C; }

extern "C" gdr_status_t gdr_layer_norm_fwd(int64_t R, int64_t C, gdr_dtype_t in_dt, const void* x,
                                           int64_t x_stride, gdr_dtype_t res_dt, const void* res,
                                           int64_t res_stride, const float* w, const float* b,
                                           float eps, gdr_dtype_t out_dt, void* y, void* h,
                                           hipStream_t stream) {
    const gdr_status_t st = norm_check(R, C, in_dt, res_dt, out_dt, eps);
    if (st != GDR_OK) return st;
    const int64_t s[2] = {x_stride, res_stride};
    if (!strides_ok(s, 2)) return GDR_ERR_INVALID;
    if (R == 0 || C == 0) return GDR_OK;
    if (!elem_ok(x, elem(in_dt)) || !elem_ok(y, elem(out_dt)) || !opt_elem(w, 4) ||
        !opt_elem(b, 4) || !opt_elem(res, elem(res_dt)) || (res && !elem_ok(h, elem(res_dt))))
        return GDR_ERR_INVALID;
    if (norm_fwd_work_items(R, C) > (double)kMaxWorkItems) return GDR_ERR_INVALID;
    // y may be x and h may be res
    if (!apart({y, res ? h : nullptr}, {w, b}) || !apart({y}, {res}) ||
        (res && !apart({h}, {x})))
        return GDR_ERR_INVALID;
    if (y == x && (in_dt != out_dt || !packed(R, C, x_stride))) return GDR_ERR_INVALID;
    if (res && h == res && !packed(R, C, res_stride)) return GDR_ERR_INVALID;
    NormArgs a{};
    a.R = R;
    a.C = C;
    a.in_bf16 = in_dt == GDR_BF16;
    a.res_bf16 = res_dt == GDR_BF16;
    a.out_bf16 = out_dt == GDR_BF16;
    a.x = x;
    a.res = res;
    a.xr = x_stride;
    a.rr = res_stride;
    a.w = w;
    a.b = b;
    a.eps = eps;
    a.y = y;
    a.h = h;
    a.stream = stream;
    return from_hip(launch_norm_fwd(a));
}

extern "C" size_t gdr_layer_norm_bwd_workspace_size(int64_t R, int64_t C) {
    if (R <= 0 || C <= 0 || norm_check(R, C, GDR_F32, GDR_F32, GDR_F32, 0.f) != GDR_OK) return 0;
    return norm_bwd_workspace_bytes(R, C);
}

extern "C" gdr_status_t gdr_layer_norm_bwd(int64_t R, int64_t C, gdr_dtype_t in_dt, const void* x,
                                           int64_t x_stride, const float* w, gdr_dtype_t dy_dt,
                                           const void* dy, int64_t dy_stride, float eps,
                                           gdr_dtype_t grad_dt, const void* dres,
                                           int64_t dres_stride, void* dx, float* dw, float* db,
                                           void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
    const gdr_status_t st = norm_check(R, C, in_dt, dy_dt, grad_dt, eps);
    if (st != GDR_OK) return st;
    const int64_t s[3] = {x_stride, dy_stride, dres_stride};
    if (!strides_ok(s, 3)) return GDR_ERR_INVALID;
    if (C == 0) return GDR_OK;
    if (!opt_elem(dw, 4) || !opt_elem(db, 4)) return GDR_ERR_INVALID;
    if (R == 0) {
        gdr_status_t e = GDR_OK;
        if (dw) e = copy_or_zero(nullptr, dw, C * 4, stream);
        if (e == GDR_OK && db) e = copy_or_zero(nullptr, db, C * 4, stream);
        return e;
    }
    if (!elem_ok(x, elem(in_dt)) || !elem_ok(dy, elem(dy_dt)) || !elem_ok(dx, elem(grad_dt)) ||
        !opt_elem(w, 4) || !opt_elem(dres, elem(grad_dt)))
        return GDR_ERR_INVALID;
    const bool sums = dw || db;
    const void* const ws = sums ? workspace : nullptr;
    if (!apart({dx, dw, db, ws}, {x, w, dy}) || !apart({dw, db, ws}, {dres}) ||
        (dres && dx == dres && !packed(R, C, dres_stride)))
        return GDR_ERR_INVALID;
    if (sums && (!ptrs_ok({workspace}) || workspace_bytes < norm_bwd_workspace_bytes(R, C)))
        return GDR_ERR_INVALID;
    NormBwdArgs a{};
    a.R = R;
    a.C = C;
    a.in_bf16 = in_dt == GDR_BF16;
    a.dy_bf16 = dy_dt == GDR_BF16;
    a.grad_bf16 = grad_dt == GDR_BF16;
    a.x = x;
    a.dy = dy;
    a.dres = dres;
    a.xr = x_stride;
    a.yr = dy_stride;
    a.rr = dres_stride;
    a.w = w;
    a.eps = eps;
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.stream = stream;
    return from_hip(launch_norm_bwd(a));
}

static bool ssm_sizes_ok(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    if (B < 0 || T < 0 || D < 0 || G < 1 || N < 1) return false;
    if (D % G != 0) return false;
    // offsets stay far below 2^63: the kept states take at most 4 floats per
    // state (N = 1) and 8 tokens, the partials of dB and dC at most 8 per element
    // of Bm and block of 64 channels
    return conv_sizes_ok(B, T, D) && (double)B * (double)T * (double)D * (double)N < 1.0e16 &&
           (double)B * (double)(T + 64) * (double)G * (double)N < 1.0e16;
}

static gdr_status_t ssm_check(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N,
                              gdr_dtype_t in_dt, gdr_dtype_t other_dt, uint32_t flags) {
    if (!ssm_sizes_ok(B, T, D, G, N)) return GDR_ERR_INVALID;
    if (!dtype_ok(in_dt) || !dtype_ok(other_dt)) return GDR_ERR_UNSUPPORTED;
    if (N > GDR_SSM_MAX_N || (flags & ~GDR_SSM_SOFTPLUS)) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Fills the fields that the forward, the token and the backward share.
template <typename Args>
static void ssm_fill(Args& a, int64_t B, int64_t T, int64_t D, int64_t G, int64_t N,
                     gdr_dtype_t in_dt, const void* x, const void* dt, const float* A,
                     const void* Bm, const void* Cm, const float* D_skip, const void* z,
                     const float* dt_bias, const float* h0, uint32_t flags,
                     const int64_t* strides) {
    a.B = B;
    a.T = T;
    a.D = D;
    a.G = G;
    a.N = N;
    a.in_bf16 = in_dt == GDR_BF16;
    a.softplus = flags & GDR_SSM_SOFTPLUS;
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.Bm = Bm;
    a.Cm = Cm;
    a.D_skip = D_skip;
    a.z = z;
    a.bias = dt_bias;
    a.h0 = h0;
    pick(strides, 0, T, D, a.xb, a.xt);
    pick(strides, 1, T, D, a.dtb, a.dtt);
    pick(strides, 2, T, G * N, a.bb, a.bt);
    pick(strides, 3, T, G * N, a.cb, a.ct);
    pick(strides, 4, T, D, a.zb, a.zt);
}

static bool ssm_ptrs_ok(gdr_dtype_t in_dt, const void* x, const void* dt, const float* A,
                        const void* Bm, const void* Cm, const float* D_skip, const void* z,
                        const float* dt_bias) {
    const size_t ie = elem(in_dt);
    return elem_ok(x, ie) && elem_ok(dt, ie) && elem_ok(A, 4) && elem_ok(Bm, ie) &&
           elem_ok(Cm, ie) && opt_elem(D_skip, 4) && opt_elem(z, ie) && opt_elem(dt_bias, 4);
}

extern "C" size_t gdr_ssm_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D, int64_t G,
                                                  int64_t N) {
    if (!ssm_sizes_ok(B, T, D, G, N) || N > GDR_SSM_MAX_N || B == 0 || D == 0 || T == 0) return 0;
    return ssm_fwd_workspace_bytes(B, T, D, G, N);
}

extern "C" gdr_status_t gdr_ssm_scan_fwd(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N,
                                         gdr_dtype_t in_dt, const void* x, const void* dt,
                                         const float* A, const void* Bm, const void* Cm,
                                         const float* D_skip, const void* z, const float* dt_bias,
                                         const float* h0, const int64_t* strides, uint32_t flags,
                                         gdr_dtype_t out_dt, void* y, float* h_final,
                                         void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
    const gdr_status_t st = ssm_check(B, T, D, G, N, in_dt, out_dt, flags);
    if (st != GDR_OK) return st;
    if (!strides_ok(strides, 10)) return GDR_ERR_INVALID;
    if (B == 0 || D == 0) return GDR_OK;
    if (!opt_elem(h0, 4) || !opt_elem(h_final, 4)) return GDR_ERR_INVALID;
    if (T == 0) return h_final ? copy_or_zero(h0, h_final, B * D * N * 4, stream) : GDR_OK;
    if (!ssm_ptrs_ok(in_dt, x, dt, A, Bm, Cm, D_skip, z, dt_bias) || !elem_ok(y, elem(out_dt)))
        return GDR_ERR_INVALID;
    const SsmPlan p = ssm_fwd_plan(B, T, D, G, N);
    if (!workgroups_ok(2.0 * B * G * p.nblk * p.nseg)) return GDR_ERR_INVALID;   // 512 threads each
    const size_t need = ssm_fwd_workspace_bytes(B, T, D, G, N);
    if (need && (!ptrs_ok({workspace}) || workspace_bytes < need)) return GDR_ERR_INVALID;
    const void* const ws = need ? workspace : nullptr;
    if (!apart({y, h_final, ws}, {x, dt, A, Bm, Cm, D_skip, z, dt_bias}) || !apart({y, ws}, {h0}))
        return GDR_ERR_INVALID;
    SsmArgs a{};
    ssm_fill(a, B, T, D, G, N, in_dt, x, dt, A, Bm, Cm, D_skip, z, dt_bias, h0, flags, strides);
    a.out_bf16 = out_dt == GDR_BF16;
    a.y = y;
    a.h_final = h_final;
    a.stream = stream;
    return from_hip(launch_ssm_fwd(a, need ? static_cast<float*>(workspace) : nullptr));
}

extern "C" gdr_status_t gdr_ssm_step(int64_t Nseq, int64_t D, int64_t G, int64_t N,
                                     gdr_dtype_t in_dt, const void* x, const void* dt,
                                     const float* A, const void* Bm, const void* Cm,
                                     const float* D_skip, const void* z, const float* dt_bias,
                                     float* state, const int64_t* strides, uint32_t flags,
                                     gdr_dtype_t out_dt, void* y, hipStream_t stream) {
    const gdr_status_t st = ssm_check(Nseq, 1, D, G, N, in_dt, out_dt, flags);
    if (st != GDR_OK) return st;
    if (!strides_ok(strides, 5)) return GDR_ERR_INVALID;
    if (Nseq == 0 || D == 0) return GDR_OK;
    if (!ssm_ptrs_ok(in_dt, x, dt, A, Bm, Cm, D_skip, z, dt_bias) || !elem_ok(state, 4) ||
        !elem_ok(y, elem(out_dt)))
        return GDR_ERR_INVALID;
    if (!apart({y, state}, {x, dt, A, Bm, Cm, D_skip, z, dt_bias})) return GDR_ERR_INVALID;
    if (!workgroups_ok((double)ssm_step_workgroups(Nseq, D, N))) return GDR_ERR_INVALID;
    int64_t s[10];
    for (int i = 0; strides && i < 5; ++i) {
        s[2 * i] = strides[i];
        s[2 * i + 1] = 0;
    }
    SsmArgs a{};
    ssm_fill(a, Nseq, 1, D, G, N, in_dt, x, dt, A, Bm, Cm, D_skip, z, dt_bias, state, flags,
             strides ? s : nullptr);
    a.out_bf16 = out_dt == GDR_BF16;
    a.y = y;
    a.h_final = state;
    a.stream = stream;
    return from_hip(launch_ssm_step(a));
}

extern "C" size_t gdr_ssm_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int64_t G,
                                                  int64_t N) {
    if (!ssm_sizes_ok(B, T, D, G, N) || N > GDR_SSM_MAX_N || B == 0 || D == 0 || T == 0) return 0;
    if (!workgroups_ok((double)ssm_bwd_workgroups(B, T, D, G, N))) return 0;
    return ssm_bwd_workspace_bytes(B, T, D, G, N);
}

extern "C" gdr_status_t gdr_ssm_scan_bwd(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N,
                                         gdr_dtype_t in_dt, const void* x, const void* dt,
                                         const float* A, const void* Bm, const void* Cm,
                                         const float* D_skip, const void* z, const float* dt_bias,
                                         const float* h0, gdr_dtype_t dout_dt, const void* dout,
                                         const float* dh_final, const int64_t* strides,
                                         uint32_t flags, gdr_dtype_t grad_dt, void* dx, void* ddt,
                                         float* dA, void* dB, void* dC, float* dD, void* dz,
                                         float* ddt_bias, float* dh0, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream) {
    const gdr_status_t st = ssm_check(B, T, D, G, N, in_dt, dout_dt, flags);
    if (st != GDR_OK) return st;
    if (!dtype_ok(grad_dt)) return GDR_ERR_UNSUPPORTED;
    if (!strides_ok(strides, 12)) return GDR_ERR_INVALID;
    if (D == 0) return GDR_OK;
    if (!elem_ok(dA, 4) || !opt_elem(dD, 4) || !opt_elem(ddt_bias, 4) || !opt_elem(dh0, 4) ||
        !opt_elem(dh_final, 4) || !opt_elem(h0, 4))
        return GDR_ERR_INVALID;
    if (B == 0 || T == 0) {
        gdr_status_t e = copy_or_zero(nullptr, dA, D * N * 4, stream);
        if (e == GDR_OK && dD) e = copy_or_zero(nullptr, dD, D * 4, stream);
        if (e == GDR_OK && ddt_bias) e = copy_or_zero(nullptr, ddt_bias, D * 4, stream);
        if (e == GDR_OK && dh0 && B > 0) e = copy_or_zero(dh_final, dh0, B * D * N * 4, stream);
        return e;
    }
    const size_t ge = elem(grad_dt);
    if (!ssm_ptrs_ok(in_dt, x, dt, A, Bm, Cm, D_skip, z, dt_bias) ||
        !elem_ok(dout, elem(dout_dt)) || !elem_ok(dx, ge) || !elem_ok(ddt, ge) ||
        !elem_ok(dB, ge) || !elem_ok(dC, ge) || (z && !elem_ok(dz, ge)))
        return GDR_ERR_INVALID;
    if (!apart({dx, ddt, dA, dB, dC, dD, z ? dz : nullptr, ddt_bias, dh0, workspace},
               {x, dt, A, Bm, Cm, D_skip, z, dt_bias, h0, dout, dh_final}))
        return GDR_ERR_INVALID;
    if (!workgroups_ok((double)ssm_bwd_workgroups(B, T, D, G, N))) return GDR_ERR_INVALID;
    if (!ptrs_ok({workspace}) || workspace_bytes < ssm_bwd_workspace_bytes(B, T, D, G, N))
        return GDR_ERR_INVALID;
    SsmBwdArgs a{};
    ssm_fill(a, B, T, D, G, N, in_dt, x, dt, A, Bm, Cm, D_skip, z, dt_bias, h0, flags, strides);
    a.dout_bf16 = dout_dt == GDR_BF16;
    a.grad_bf16 = grad_dt == GDR_BF16;
    a.dout = dout;
    pick(strides, 5, T, D, a.ob, a.ot);
    a.dh_final = dh_final;
    a.dx = dx;
    a.ddt = ddt;
    a.dA = dA;
    a.dB = dB;
    a.dC = dC;
    a.dD = dD;
    a.dz = dz;
    a.dbias = ddt_bias;
    a.dh0 = dh0;
    a.stream = stream;
    return from_hip(launch_ssm_bwd(a, workspace));
}
