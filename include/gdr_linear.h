/*
 * Linear attention with a decay per head (gdr_linear_attn_*), and what its layers
 * put around it: rotary positions of q and k (gdr_rotary*) and the RMS norm in
 * front of the block, with an 8-bit output for the projections behind it
 * (gdr_rms_norm_*).  Part of libgdr.so.
 */
#ifndef GDR_LINEAR_H
#define GDR_LINEAR_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The conventions of gdr.h hold with these differences:
 *   - token tensors may be slices of wider ones.  `strides` is a HOST array of
 *     element strides, {sequence, token, head} per tensor in the order given per
 *     call (channels are always contiguous); NULL means contiguous tensors.  A
 *     stride is in [0, 2^40].  Everything without a stride is contiguous;
 *   - every pointer needs only its element's alignment (workspaces 16 bytes);
 *   - a launch has fewer than 2^32 work-items; larger calls are refused;
 *   - every sum runs in a fixed order: equal calls give equal bits;
 *   - outputs and workspaces must not overlap inputs or each other unless a call
 *     says so.  One that starts where an input or another of them starts is
 *     refused; the caller sees to the rest;
 *   - the device of the tensors must be the current device.
 */

/*
 * Linear attention with a decay per head:
 *
 *   S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,
 *
 * S a Dv x Dk fp32 matrix per sequence and head: the rule of gdr_chunk_fwd without
 * its correction, and the scan of a state space layer with one decay per head (k
 * and q its B and C, v its x times the step).
 *
 *   B, T      sequences, tokens (each >= 0)
 *   H, Hk     heads of v, g, o and the state (at most GDR_MAX_HEADS); heads of q
 *             and k, each shared by H / Hk consecutive heads (Hk divides H)
 *   Dk, Dv    multiples of 8, at most GDR_LA_MAX_D
 *   q, k      [B, T, Hk, Dk] in_dt;  v [B, T, H, Dv] in_dt; strides {q, k, v},
 *             those of tokens at most GDR_LA_MAX_TOKEN_STRIDE
 *   log_decay g, fp32: [B, T, H], or [H] with GDR_LA_HEAD_DECAY, or NULL (no
 *             decay).  Meant to be <= 0; minus infinity (anything below -10000)
 *             forgets all tokens before, as at the first token of a packed
 *             sequence
 *   s0        [B, H, Dv, Dk] fp32 or NULL (zeros)
 *   o         [B, T, H, Dv] out_dt
 *   s_final   [B, H, Dv, Dk] fp32 or NULL; may be s0 itself
 *   workspace states of a sequence's segments, where few long sequences run as
 *             segments side by side, and room for a copy of s0 (which s_final's store
 *             would meet there); may be NULL when its size is 0
 *
 * fp32 inputs are computed in fp32.  bf16 inputs run on the bf16 matrix cores with
 * fp32 accumulation; every computed operand enters as three bf16 terms, so products
 * carry the 24 bits of fp32 (two terms, 2^-17 of the operand, in products that only a
 * bf16 o, dq, dk or dv takes).  Decays come from sums in 64 bits.  A value that
 * is infinite or no number reaches no token before it; the state that it enters has no
 * numbers from then on, behind a decay of 0 too (0 times it).
 */
#define GDR_LA_HEAD_DECAY 1u
#define GDR_LA_MAX_D 128
#define GDR_LA_MAX_TOKEN_STRIDE 8388608

size_t gdr_linear_attn_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv,
                                          gdr_dtype_t in_dt);

gdr_status_t gdr_linear_attn_fwd(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk,
                                 int64_t Dv, gdr_dtype_t in_dt, const void *q, const void *k,
                                 const void *v, const int64_t *strides, const float *log_decay,
                                 const float *s0, float scale, uint32_t flags, gdr_dtype_t out_dt,
                                 void *o, float *s_final, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* One decode token of N sequences: q, k [N, Hk, Dk], v [N, H, Dv] (strides
 * {sequence, head} each), log_decay [N, H] or [H] or NULL, the state [N, H, Dv, Dk]
 * moved on in place, o [N, H, Dv]. */
gdr_status_t gdr_linear_attn_step(int64_t N, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                                  gdr_dtype_t in_dt, const void *q, const void *k, const void *v,
                                  const int64_t *strides, const float *log_decay, float *state,
                                  float scale, uint32_t flags, gdr_dtype_t out_dt, void *o,
                                  hipStream_t stream);

/*
 * Reverse mode of gdr_linear_attn_fwd: dout [B, T, H, Dv] in_dt is the gradient of
 * o, ds_final [B, H, Dv, Dk] fp32 or NULL that of s_final; strides {q, k, v, dout}.
 * Writes dq, dk [B, T, Hk, Dk] (sums over the heads that share one: zeros where H is
 * 0) and dv [B, T, H, Dv] in grad_dt, and in fp32 dlog_decay (shaped as log_decay;
 * NULL: not wanted, as without log_decay; 0 where the decay itself is 0, which also
 * keeps packed sequences' gradients apart) and ds0 [B, H, Dv, Dk] (or NULL).  The
 * workspace holds states at every 512 tokens (with GDR_LA_HEAD_DECAY 256) or fewer (at
 * most twice 4 B H Dv Dk bytes each; twice that where a sequence runs as segments),
 * 8 B T H ceil(Dk / 16) bytes for the decay's gradient and, where Hk < H, 8 B T H Dk
 * bytes for dq and dk of each head.
 * A value that is infinite or no number is in the gradients that have it in their sums
 * and in no others, with one exception: one of k or v is also in dlog_decay of the tokens
 * before it, back to a decay of 0 or at most as far as the kept states are apart.
 * Workspace sizes are 0 for arguments the calls reject.
 */
size_t gdr_linear_attn_bwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk,
                                          int64_t Dv, gdr_dtype_t in_dt, uint32_t flags);

gdr_status_t gdr_linear_attn_bwd(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk,
                                 int64_t Dv, gdr_dtype_t in_dt, const void *q, const void *k,
                                 const void *v, const int64_t *strides, const float *log_decay,
                                 const float *s0, const void *dout, const float *ds_final,
                                 float scale, uint32_t flags, gdr_dtype_t grad_dt, void *dq,
                                 void *dk, void *dv, float *dlog_decay, float *ds0,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Rotary positions of q and k: the first `rot` channels of every head as rot / 2
 * pairs (a, b), turned by angle_i = position freqs[i] and scaled:
 *
 *   (a, b) -> scale (a cos - b sin, a sin + b cos).
 *
 * Pair i is channels i and i + rot / 2, or 2 i and 2 i + 1 with
 * GDR_ROTARY_INTERLEAVED.  The other channels are copied.  GDR_ROTARY_INVERSE turns
 * back: the reverse mode, for the gradients of the outputs.
 *
 *   q, k      [B, T, Hq, D], [B, T, Hk, D] dt (k NULL with Hk = 0); strides
 *             {q, k, q_out, k_out}; Hq + Hk at most GDR_MAX_HEADS
 *   rot       even, 0 < rot <= D <= GDR_ROTARY_MAX_D
 *   positions [B, T] int64 with pos_stride elements from sequence to sequence
 *             (0: shared), or NULL: start + t
 *   freqs     [rot / 2] double (device), as from gdr_rotary_frequencies
 *   q_out, k_out  like q and k, their heads at places of their own (each stride
 *             passes what the smaller ones span); may be q and k themselves with
 *             equal strides
 *
 * Sine and cosine are within 2^-22 at every position (whole numbers up to 2^53, beyond
 * as the nearest double) while |position freqs[i]| is at most 2^48: the angle is formed
 * and reduced in two doubles.
 */
#define GDR_ROTARY_INTERLEAVED 1u
#define GDR_ROTARY_INVERSE 2u
#define GDR_ROTARY_MAX_D 1024

gdr_status_t gdr_rotary(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t rot,
                        gdr_dtype_t dt, const void *q, const void *k, const int64_t *strides,
                        const int64_t *positions, int64_t pos_stride, int64_t start,
                        const double *freqs, float scale, uint32_t flags, void *q_out,
                        void *k_out, hipStream_t stream);

/*
 * The rates base^{-2 i / rot} in HOST memory [rot / 2], scaled for contexts `factor`
 * times longer than the `original` tokens of training:
 *
 *   GDR_ROTARY_PLAIN     as they are
 *   GDR_ROTARY_LINEAR    all divided by factor (positions interpolated)
 *   GDR_ROTARY_BASE      base multiplied by factor^{rot / (rot - 2)}, which divides
 *                        the slowest by factor and leaves the fastest
 *   GDR_ROTARY_PARTS     by the turns r = original rate / 2 pi that a rate makes in
 *                        training: divided by factor up to `low` turns, left from
 *                        `high` on, in between rate (w + (1 - w) / factor) with
 *                        w = (r - low) / (high - low)
 */
typedef enum {
    GDR_ROTARY_PLAIN = 0,
    GDR_ROTARY_LINEAR = 1,
    GDR_ROTARY_BASE = 2,
    GDR_ROTARY_PARTS = 3
} gdr_rotary_scaling_t;

gdr_status_t gdr_rotary_frequencies(int64_t rot, double base, gdr_rotary_scaling_t scaling,
                                    double factor, double low, double high, double original,
                                    double *freqs);

/*
 * RMS norm of R rows of C channels (C up to GDR_RMS_MAX_C), with the residual
 * stream's sum in front of it when `res` is given:
 *
 *   h = x + res (rounded to res_dt, written out and normalised as written), or x;
 *   y = h / sqrt(mean h^2 + eps) w.
 *
 * The squares are summed in fp32: a row whose sum is infinite there (with an infinite
 * value, or values above 2^64 / sqrt(C)) is divided by infinity, to zeros and, for
 * infinite values, to what is no number.  A row with a value that is no number has no
 * others in y.
 *
 *   R         fewer than 2^24, with C between 8193 and 16384 than 2^23
 *   x, res, h, w, eps, y   as for gdr_layer_norm_fwd (gdr_block.h): y may be x, h
 *                          may be res
 */
#define GDR_RMS_MAX_C 1048576

gdr_status_t gdr_rms_norm_fwd(int64_t R, int64_t C, gdr_dtype_t in_dt, const void *x,
                              int64_t x_stride, gdr_dtype_t res_dt, const void *res,
                              int64_t res_stride, const float *w, float eps, gdr_dtype_t out_dt,
                              void *y, void *h, hipStream_t stream);

/*
 * The same with y in 8 bits: per row (group 0) or group of 32, 64 or 128 channels
 * (which divides C), scale = max |y| / 448 (GDR_Q_E4M3, the finite-only 8-bit float
 * with 3 bits of mantissa) or / 127 (GDR_Q_INT8), q = y / scale (both in fp32, and
 * their quotient) rounded to nearest even.  scales [R, C / group] ([R, 1]) fp32; y [R, C]
 * bytes.  A scale below fp32's normal numbers is written as 0 with zeros.  Where y has a
 * value that is no number (see above), its group's or row's scale is none either; the
 * other groups of a row with an infinite value have scales of 0 and zeros.
 */
typedef enum { GDR_Q_E4M3 = 0, GDR_Q_INT8 = 1 } gdr_q8_t;

gdr_status_t gdr_rms_norm_quant(int64_t R, int64_t C, gdr_dtype_t in_dt, const void *x,
                                int64_t x_stride, gdr_dtype_t res_dt, const void *res,
                                int64_t res_stride, const float *w, float eps, gdr_q8_t type,
                                int64_t group, void *y, float *scales, void *h,
                                hipStream_t stream);

/*
 * Reverse mode: x is the normalised tensor (h where a residual was added), dy
 * [R, C] dy_dt the gradient of y.  Writes dx [R, C] grad_dt (plus dres [R, C]
 * grad_dt, the gradient that reaches h past the norm, when given; dx may be dres
 * itself with dres_stride == C or one row) and dw [C] fp32 (or NULL).  The workspace
 * (partial sums) may be NULL when dw is.  Its size is 0 for arguments the call
 * rejects.
 */
size_t gdr_rms_norm_bwd_workspace_size(int64_t R, int64_t C);

gdr_status_t gdr_rms_norm_bwd(int64_t R, int64_t C, gdr_dtype_t in_dt, const void *x,
                              int64_t x_stride, const float *w, gdr_dtype_t dy_dt, const void *dy,
                              int64_t dy_stride, float eps, gdr_dtype_t grad_dt, const void *dres,
                              int64_t dres_stride, void *dx, float *dw, void *workspace,
                              size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_LINEAR_H */
