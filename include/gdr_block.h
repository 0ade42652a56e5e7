/*
 * Operators around the token mixer: the short causal convolution before it
 * (gdr_short_conv_*), the selective state space scan beside it (gdr_ssm_*),
 * and the layer norm in front of the block (gdr_layer_norm_*), forward and
 * backward, the first two also for one decode token.  Part of libgdr.so.
 */
#ifndef GDR_BLOCK_H
#define GDR_BLOCK_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The conventions of gdr.h hold with these differences:
 *   - token tensors may be slices of wider ones.  `strides` is a HOST array
 *     of element strides, {sequence, token} per tensor in the order given per
 *     call (channels are always contiguous); NULL means contiguous tensors.
 *     A stride is in [0, 2^40].  Everything without a stride is contiguous;
 *   - every pointer needs only its element's alignment (workspaces 16 bytes);
 *   - sizes are free: channels, lengths and states of any count within the
 *     stated limits, no multiple of anything.  A launch has fewer than 2^32
 *     work-items, in workgroups of 256 (the scan's of up to 512); larger calls
 *     are refused.  Layer norm counts a workgroup per row, forward of 512 from
 *     8193 to 16384 channels: fewer than 2^24 rows, there fewer than 2^23;
 *   - the gradients of activations are written in grad_dt (GDR_F32 or
 *     GDR_BF16), those of parameters and states in fp32.  Every sum runs in a
 *     fixed order: equal calls give equal bits;
 *   - outputs and workspaces must not overlap inputs or each other unless a
 *     call says so.  One that starts where an input or another of them starts
 *     is refused; the caller sees to the rest;
 *   - the device of the tensors must be the current device.
 */

/*
 * Short causal depthwise convolution, the step of the block's q, k and v
 * paths between projection and mixer (review of GDN on
 * meaningful96.github.io, section 3.8), per channel c:
 *
 *   u_t = bias + sum_{j < K} w[c][j] x_{t - K + 1 + j},   y_t = u_t or, with
 *   GDR_CONV_SILU, u_t sigmoid(u_t);
 *
 * x before the sequence is the state s0: its last K - 1 inputs, oldest first.
 *
 *   B, T, C   sequences, tokens, channels (each >= 0);  K in {2, 3, 4}
 *   x         [B, T, C] in_dt; strides {x}
 *   w, bias   [C, K] and [C] fp32; bias NULL means 0
 *   s0        [B, K - 1, C] in_dt or NULL (zeros)
 *   y         [B, T, C] out_dt
 *   s_final   [B, K - 1, C] in_dt or NULL: the last K - 1 rows of [s0; x],
 *             bit for bit; may be s0 itself
 *
 * Sums in fp32.
 */
#define GDR_CONV_SILU 1u

gdr_status_t gdr_short_conv_fwd(int64_t B, int64_t T, int64_t C, int64_t K,
                                gdr_dtype_t in_dt, const void *x,
                                const int64_t *strides, const float *w,
                                const float *bias, const void *s0,
                                uint32_t flags, gdr_dtype_t out_dt, void *y,
                                void *s_final, hipStream_t stream);

/* One decode token of N sequences: x [N, C] with a stride per sequence, the
 * state [N, K - 1, C] in_dt moved on in place, y [N, C]. */
gdr_status_t gdr_short_conv_step(int64_t N, int64_t C, int64_t K,
                                 gdr_dtype_t in_dt, const void *x,
                                 int64_t x_stride, const float *w,
                                 const float *bias, void *state,
                                 uint32_t flags, gdr_dtype_t out_dt, void *y,
                                 hipStream_t stream);

/*
 * Reverse mode of gdr_short_conv_fwd.  dy [B, T, C] dy_dt (strides {x, dy}),
 * ds_final [B, K - 1, C] fp32 or NULL (gradient of s_final).  Writes dx
 * [B, T, C] grad_dt, dw [C, K], dbias [C] and ds0 [B, K - 1, C] fp32; each of
 * dw, dbias, ds0 may be NULL.  The workspace (partial sums of dw and dbias)
 * may be NULL when both are.  Its size is 0 for arguments the call rejects.
 */
size_t gdr_short_conv_bwd_workspace_size(int64_t B, int64_t T, int64_t C,
                                         int64_t K);

gdr_status_t gdr_short_conv_bwd(int64_t B, int64_t T, int64_t C, int64_t K,
                                gdr_dtype_t in_dt, const void *x,
                                const float *w, const float *bias,
                                const void *s0, gdr_dtype_t dy_dt,
                                const void *dy, const int64_t *strides,
                                const float *ds_final, uint32_t flags,
                                gdr_dtype_t grad_dt, void *dx, float *dw,
                                float *dbias, float *ds0, void *workspace,
                                size_t workspace_bytes, hipStream_t stream);

/*
 * Selective state space scan, the diagonal recurrent mixer of hybrid stacks.
 * Per channel d of group g = d / (D / G), with N states:
 *
 *   Delta_t = softplus(dt_t + dt_bias)   (GDR_SSM_SOFTPLUS; else their sum),
 *   h_t[n] = exp(Delta_t A[d][n]) h_{t-1}[n] + Delta_t x_t B_t[g][n],
 *   y_t = sum_n C_t[g][n] h_t[n] + D_skip[d] x_t,  times z_t sigmoid(z_t)
 *   when z is given.
 *
 *   B, T, D   sequences, tokens, channels (each >= 0)
 *   G         groups of channels that share Bm and Cm; divides D
 *   N         states per channel, 1 to GDR_SSM_MAX_N
 *   x, dt, z  [B, T, D] in_dt; z may be NULL
 *   Bm, Cm    [B, T, G, N] in_dt, [G, N] contiguous
 *   strides   {x, dt, Bm, Cm, z}
 *   A         [D, N] fp32, <= 0 in use (not checked).  -inf and values below
 *             -2.36e38 act as -2.36e38: any Delta above 1e-36 forgets at once
 *   D_skip, dt_bias  [D] fp32 or NULL (zeros)
 *   h0        [B, D, N] fp32 or NULL (zeros)
 *   y         [B, T, D] out_dt
 *   h_final   [B, D, N] fp32 or NULL; may be h0 itself
 *
 * fp32 throughout.  Where B D leaves most of the chip idle the sequence runs
 * as segments side by side, whose states go through the workspace (size 0:
 * none needed, and for arguments the call rejects).
 */
#define GDR_SSM_SOFTPLUS 1u
#define GDR_SSM_MAX_N 64

size_t gdr_ssm_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D,
                                       int64_t G, int64_t N);

gdr_status_t gdr_ssm_scan_fwd(int64_t B, int64_t T, int64_t D, int64_t G,
                              int64_t N, gdr_dtype_t in_dt, const void *x,
                              const void *dt, const float *A, const void *Bm,
                              const void *Cm, const float *D_skip,
                              const void *z, const float *dt_bias,
                              const float *h0, const int64_t *strides,
                              uint32_t flags, gdr_dtype_t out_dt, void *y,
                              float *h_final, void *workspace,
                              size_t workspace_bytes, hipStream_t stream);

/* One decode token of Nseq sequences: the tensors above without T (strides:
 * one per tensor, {x, dt, Bm, Cm, z}), state [Nseq, D, N] fp32 in place. */
gdr_status_t gdr_ssm_step(int64_t Nseq, int64_t D, int64_t G, int64_t N,
                          gdr_dtype_t in_dt, const void *x, const void *dt,
                          const float *A, const void *Bm, const void *Cm,
                          const float *D_skip, const void *z,
                          const float *dt_bias, float *state,
                          const int64_t *strides, uint32_t flags,
                          gdr_dtype_t out_dt, void *y, hipStream_t stream);

/*
 * Reverse mode of gdr_ssm_scan_fwd: dout [B, T, D] dout_dt is the gradient of
 * y, dh_final [B, D, N] fp32 or NULL that of h_final; strides
 * {x, dt, Bm, Cm, z, dout}.  Writes dx, ddt [B, T, D], dB, dC [B, T, G, N]
 * and dz [B, T, D] (NULL without z) in grad_dt, and in fp32 dA [D, N], dD and
 * ddt_bias [D] and dh0 [B, D, N] (each of the last three may be NULL).
 * Without channels (D == 0) nothing is launched, as in every call: dB and dC,
 * which have elements even then, are the caller's to clear.  The states are
 * run again from the inputs; the workspace holds one state in S tokens and the
 * partial sums, mainly 4 B T P (D / S + 2 G ceil(D / (64 G))) bytes, where P is
 * N rounded up to 4, 8, 16, 32 or 64 and S = 8, 8, 16, 8 or 4.  Its size is 0
 * for arguments the call rejects.
 */
size_t gdr_ssm_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D,
                                       int64_t G, int64_t N);

gdr_status_t gdr_ssm_scan_bwd(int64_t B, int64_t T, int64_t D, int64_t G,
                              int64_t N, gdr_dtype_t in_dt, const void *x,
                              const void *dt, const float *A, const void *Bm,
                              const void *Cm, const float *D_skip,
                              const void *z, const float *dt_bias,
                              const float *h0, gdr_dtype_t dout_dt,
                              const void *dout, const float *dh_final,
                              const int64_t *strides, uint32_t flags,
                              gdr_dtype_t grad_dt, void *dx, void *ddt,
                              float *dA, void *dB, void *dC, float *dD,
                              void *dz, float *ddt_bias, float *dh0,
                              void *workspace, size_t workspace_bytes,
                              hipStream_t stream);

/*
 * Layer norm of R rows of C channels (C up to GDR_NORM_MAX_C), with the
 * residual stream's sum in front of it when `res` is given:
 *
 *   h = x + res (rounded to res_dt, written out and normalised as written),
 *   or x;   y = (h - mean h) / sqrt(mean (h - mean h)^2 + eps) w + b.
 *
 *   x         [R, C] in_dt, x_stride elements from row to row
 *   res, h    [R, C] res_dt, res with res_stride; both NULL without residual.
 *             h may be res itself (with res_stride == C, or one row)
 *   w, b      [C] fp32 or NULL (ones, zeros)
 *   y         [R, C] out_dt; may be x itself (same dtype, x_stride == C or one
 *             row)
 *   eps       >= 0
 *
 * Statistics in fp32, the variance from centred values.
 */
#define GDR_NORM_MAX_C 1048576

gdr_status_t gdr_layer_norm_fwd(int64_t R, int64_t C, gdr_dtype_t in_dt,
                                const void *x, int64_t x_stride,
                                gdr_dtype_t res_dt, const void *res,
                                int64_t res_stride, const float *w,
                                const float *b, float eps, gdr_dtype_t out_dt,
                                void *y, void *h, hipStream_t stream);

/*
 * Reverse mode: x is the normalised tensor (h where a residual was added), dy
 * [R, C] dy_dt the gradient of y.  Writes dx [R, C] grad_dt (plus dres
 * [R, C] grad_dt, the gradient that reaches h past the norm, when given; dx
 * may be dres itself with dres_stride == C or one row) and dw, db [C] fp32,
 * each of which may be NULL.  The workspace (partial sums) may be NULL when
 * both are.  Its size is 0 for arguments the call rejects.
 */
size_t gdr_layer_norm_bwd_workspace_size(int64_t R, int64_t C);

gdr_status_t gdr_layer_norm_bwd(int64_t R, int64_t C, gdr_dtype_t in_dt,
                                const void *x, int64_t x_stride,
                                const float *w, gdr_dtype_t dy_dt,
                                const void *dy, int64_t dy_stride, float eps,
                                gdr_dtype_t grad_dt, const void *dres,
                                int64_t dres_stride, void *dx, float *dw,
                                float *db, void *workspace,
                                size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_BLOCK_H */
