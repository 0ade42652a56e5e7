// Arguments and launchers of the operators around the token mixer.
#pragma once

#include "launch.h"

namespace gdr {

// Short causal convolution, all directions.  x and dy are rows of C channels
// with a stride per sequence (xb, yb) and per token (xt, yt); everything else
// is contiguous.  s0 and s_final [B, K - 1, C] in the input dtype.
struct ConvArgs {
    int64_t B, T, C;
    int K;
    bool in_bf16, out_bf16, dy_bf16, grad_bf16;
    bool silu;
    const void* x;
    int64_t xb, xt;
    const float *w, *bias;
    const void* s0;
    void *y, *s_final;
    // backward
    const void* dy;
    int64_t yb, yt;
    const float* ds_final;
    void* dx;
    float *dw, *dbias, *ds0;
    float* part;            // dw and dbias partials, or NULL: neither is wanted
    hipStream_t stream;
};

// Layer norm: rows of C channels, x and res with a stride per row.
struct NormArgs {
    int64_t R, C;
    bool in_bf16, res_bf16, out_bf16;
    const void *x, *res;    // res NULL: no residual, no h
    int64_t xr, rr;
    const float *w, *b;
    float eps;
    void *y, *h;
    hipStream_t stream;
};

struct NormBwdArgs {
    int64_t R, C;
    bool in_bf16, dy_bf16, grad_bf16;
    const void *x, *dy, *dres;
    int64_t xr, yr, rr;
    const float* w;
    float eps;
    void* dx;
    float *dw, *db;
    float* part;            // dw and db partials (and row statistics), or NULL
    hipStream_t stream;
};

// Selective scan forward and token: x, dt, z [B, T, D] and Bm, Cm
// [B, T, G, N] with strides per sequence and token.  hend and sdelta: see
// ssm_fwd_kernel.
struct SsmArgs {
    int64_t B, T, D, G, N;
    bool in_bf16, out_bf16, softplus;
    const void *x, *dt, *Bm, *Cm, *z;
    int64_t xb, xt, dtb, dtt, bb, bt, cb, ct, zb, zt;
    const float *A, *D_skip, *bias, *h0;
    void* y;
    float* h_final;
    float *hend, *sdelta;
    hipStream_t stream;
};

struct SsmBwdArgs {
    int64_t B, T, D, G, N;
    bool in_bf16, dout_bf16, grad_bf16, softplus;
    const void *x, *dt, *Bm, *Cm, *z, *dout;
    int64_t xb, xt, dtb, dtt, bb, bt, cb, ct, zb, zt, ob, ot;
    const float *A, *D_skip, *bias, *h0, *dh_final;
    void *dx, *ddt, *dB, *dC, *dz;
    float *dA, *dD, *dbias, *dh0;
    // workspace: kept states and their sums of Delta, the segments' end
    // states, start gradients and sums of Delta, partials of the parameters'
    // gradients and of dB, dC
    float *ckpt, *csum, *hend, *gstart, *sdelta, *part, *bcpart;
    hipStream_t stream;
};

// Launch shape of a scan: channel blocks per group,
// segments per sequence and their length.
struct SsmPlan {
    int64_t nblk, nseg, L;
};

hipError_t launch_conv_fwd(const ConvArgs& a);
hipError_t launch_conv_step(const ConvArgs& a);      // T = 1; s0 and s_final the state
hipError_t launch_conv_bwd(const ConvArgs& a);
size_t conv_bwd_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t K);
int64_t conv_workgroups(int64_t B, int64_t T, int64_t C);
hipError_t launch_norm_fwd(const NormArgs& a);
hipError_t launch_norm_bwd(const NormBwdArgs& a);
double norm_fwd_work_items(int64_t R, int64_t C);
size_t norm_bwd_workspace_bytes(int64_t R, int64_t C);
int64_t ssm_padded_states(int64_t N);
int64_t ssm_most_segments(int64_t T);
int64_t ssm_step_workgroups(int64_t B, int64_t D, int64_t N);
SsmPlan ssm_fwd_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N);
size_t ssm_fwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N);
hipError_t launch_ssm_fwd(SsmArgs a, float* ws);
hipError_t launch_ssm_step(const SsmArgs& a);        // h0 and h_final the state
size_t ssm_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N);
int64_t ssm_bwd_workgroups(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N);
hipError_t launch_ssm_bwd(SsmBwdArgs a, void* ws);
// out[m] = sum_p part[p][m] over P rows of M columns, cut into two outputs of m0
// and M - m0 columns (either may be NULL).
hipError_t launch_sum_partials(const float* part, int64_t P, int64_t M, float* o0, int64_t m0,
                               float* o1, hipStream_t st);

}  // namespace gdr
