// Arguments and launchers of linear attention, rotary positions and RMS norm.
#pragma once

#include "launch.h"

namespace gdr {

// A token tensor [B, T, heads, channels] with element strides per sequence, token
// and head; `share` heads of the call read one head of it.
struct LaTensor {
    const void* p;
    int64_t sb, st, sh;
    int64_t share;
};

// One chain over the tokens of every (sequence, head), forwards or backwards:
//
//   H_t = e^{g} H_{t-1} + upd z_t y_t^T,
//   out_t = pair sum_{j <= t} e^{..} (x_t . y_j) z_j + inter e^{..} H_start x_t
//
// with kd channels of x and y, zd of z and out.  The state [zd, kd] lies with
// strides hz, hk inside each (sequence, head)'s Dk Dv floats.
struct LaJob {
    LaTensor x, y, z;
    int kd, zd;
    bool back;
    float pair, inter, upd;
    // out [B, T, H, zd] or [B, T, H / share, zd]
    void* out;
    int64_t ob, ot, oh;
    bool out_bf16;
    // states: start [B, H, ..] of the chain (NULL: zeros), and of its segments behind
    // the first [slot, B, H, ..], h_step slots a segment, the last of each the state
    // between it and the next (backwards: the one before); end [B, H, ..] (for the
    // states alone: the own ones of all segments but the last [.., B, H, ..], as from
    // zeros, their decays in seg_decay)
    const float *h_in, *h_seg;
    int64_t h_step;
    float* h_out;
    float* seg_decay;
    int64_t hz, hk;
    bool end_decay;         // the end also goes through the first token's decay
    // states kept at every `every` tokens, [block, B, H, ...]: after tokens
    // forwards, before them backwards; NULL: none
    float* keep;
    bool keep_end;          // forwards: the end too
    // dots[slot][B][T][H]: out_t . r_t over 16 channels each; NULL: none
    LaTensor r;
    float* dots;
};

struct LaChain {
    int64_t B, T, H;
    int64_t L, nseg;        // tokens per segment, segments
    int64_t every;
    bool bf16;
    const float* g;         // log decay [B, T, H], or [H] with g_head, or NULL
    bool g_head;
    int64_t state;          // Dk Dv
    int njobs;
    LaJob job[3];
    hipStream_t stream;
};

struct LaArgs {
    int64_t B, T, H, Hk, Dk, Dv;
    bool bf16;
    LaTensor q, k, v;
    const float* g;
    bool g_head;
    const float* s0;
    float scale;
    hipStream_t stream;
    // forward
    bool out_bf16;
    void* o;
    float* s_final;
    // backward
    LaTensor dout;
    const float* ds_final;
    bool grad_bf16;
    void *dq, *dk, *dv;
    float *dg, *ds0;
    void* workspace;
};

struct LaStepArgs {
    int64_t N, H, Hk, Dk, Dv;
    bool bf16, out_bf16;
    LaTensor q, k, v;
    const float* g;
    bool g_head;
    float scale;
    float* state;
    void* o;
    hipStream_t stream;
};

// q or k of the rotary call, in and out, with strides per sequence, token, head.
struct RotarySide {
    const void* in;
    void* out;
    int64_t ib, it, ih, ob, ot, oh;
};

struct RotaryArgs {
    int64_t B, T, Hq, Hk, D, rot;
    bool bf16, interleaved, inverse;
    RotarySide q, k;
    const int64_t* positions;   // NULL: start + t
    int64_t pos_stride, start;
    const double* freqs;
    float scale;
    hipStream_t stream;
    // by rotary_shape: units of 8 channels per head, those that turn first; tokens
    // per workgroup
    int units, turning, tokens;
};

// RMS norm: rows of C channels, x and res with a stride per row.
struct RmsArgs {
    int64_t R, C;
    bool in_bf16, res_bf16, out_bf16;
    const void *x, *res;        // res NULL: no residual, no h
    int64_t xr, rr;
    const float* w;
    float eps;
    void *y, *h;
    int q8;                     // 0: y in fp32 or bf16; 1: e4m3; 2: int8
    int64_t group;              // channels per scale (C: the row)
    float* scales;
    hipStream_t stream;
};

struct RmsBwdArgs {
    int64_t R, C;
    bool in_bf16, dy_bf16, grad_bf16;
    const void *x, *dy, *dres;
    int64_t xr, yr, rr;
    const float* w;
    float eps;
    void* dx;
    float* dw;
    float* part;                // partial sums of dw (and the rows' rstd), or NULL
    hipStream_t stream;
};

void rotary_shape(RotaryArgs& a);
double rotary_work_items(const RotaryArgs& a);
hipError_t launch_rotary(const RotaryArgs& a);
double rms_work_items(int64_t R, int64_t C);
hipError_t launch_rms_fwd(const RmsArgs& a);
size_t rms_bwd_workspace_bytes(int64_t R, int64_t C);
hipError_t launch_rms_bwd(const RmsBwdArgs& a);

int64_t la_fwd_workgroups(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, bool bf16);
size_t la_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, bool bf16);
hipError_t launch_la_fwd(const LaArgs& a);
int64_t la_bwd_workgroups(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, bool bf16,
                          bool g_head);
size_t la_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                              bool bf16, bool g_head);
hipError_t launch_la_bwd(const LaArgs& a);
hipError_t launch_la_step(const LaStepArgs& a);
int64_t la_step_workgroups(int64_t N, int64_t H, int64_t Dk, int64_t Dv);

}  // namespace gdr
