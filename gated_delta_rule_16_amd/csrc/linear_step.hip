// gdr_linear_attn_step: one decode token of linear attention, state in place.
//
// Row i of the state (value channel i) meets only itself, v_i and the shared k, q
// and decay: s_i <- e^g s_i + v_i k, o_i = scale s_i . q, one pass over each row.
// Bound by HBM: every (sequence, head) streams Dv x Dk fp32 in and out.  A row is
// read by 16 lanes (Dk up to 64) or 32, 16 bytes each; a wave has all of its rows'
// loads in flight before any arithmetic, and the traffic is non-temporal (256
// sequences, 16 heads of 128 x 128: 96 us, 5.6 TB/s).
#include "linear_launch.h"
#include "mfma_common.h"
#include "rows.h"

namespace gdr {

namespace {

constexpr int ROWS = 64;        // state rows per workgroup

__device__ __forceinline__ const char* base_of(const LaTensor& t, int64_t n, int64_t h,
                                               size_t elem) {
    return static_cast<const char*>(t.p) + (n * t.sb + h / t.share * t.sh) * elem;
}

template <int LPR, bool BF16>
__global__ __launch_bounds__(256) void la_step_kernel(LaStepArgs a, int nb) {
    constexpr int RPP = 64 / LPR, PASSES = ROWS / 4 / RPP;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t nh = blockIdx.x / nb, h = nh % a.H, n = nh / a.H;
    const int row0 = (int)(blockIdx.x % nb) * ROWS + wv * (ROWS / 4) + lane / LPR;
    const int c = lane % LPR * 4;
    constexpr size_t es = BF16 ? 2 : 4;
    float* S = a.state + nh * (a.Dk * a.Dv);
    const bool in = c < a.Dk;
    f32x4_e4 s[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = row0 + p * RPP;
        s[p] = f32x4_e4{0.f, 0.f, 0.f, 0.f};
        if (in && row < a.Dv)
            s[p] = __builtin_nontemporal_load(
                reinterpret_cast<const f32x4_e4*>(S + (int64_t)row * a.Dk + c));
    }
    Row<4, BF16, false> rk, rq;
    float k[4], q[4], v[PASSES];
    rk.load(base_of(a.k, n, h, es), c, in ? 4 : 0);
    rq.load(base_of(a.q, n, h, es), c, in ? 4 : 0);
    const char* vp = base_of(a.v, n, h, es);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = row0 + p * RPP;
        v[p] = 0.f;
        if (row < a.Dv) {
            if constexpr (BF16) v[p] = bf2f(reinterpret_cast<const bf16_t*>(vp)[row]);
            else v[p] = reinterpret_cast<const float*>(vp)[row];
        }
    }
    float d = 1.f;
    if (a.g) d = expf(a.g_head ? a.g[h] : a.g[nh]);
    rk.unpack(k);
    rq.unpack(q);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = row0 + p * RPP;
        float o = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[p][e] = __builtin_fmaf(v[p], k[e], s[p][e] * d);
            o = __builtin_fmaf(s[p][e], q[e], o);
        }
        if (in && row < a.Dv)
            __builtin_nontemporal_store(
                s[p], reinterpret_cast<f32x4_e4*>(S + (int64_t)row * a.Dk + c));
        o += dpp_mov<0xB1>(o);
        o += dpp_mov<0x4E>(o);
        o += dpp_mov<0x141>(o);
        o += dpp_mov<0x140>(o);
        if constexpr (LPR == 32) o += __shfl_xor(o, 16, 64);
        if (c == 0 && row < a.Dv) {
            const float y[1] = {o * a.scale};
            row_store<1, false>(a.o, nh * a.Dv + row, a.out_bf16, y, 1);
        }
    }
}

}  // namespace

int64_t la_step_workgroups(int64_t N, int64_t H, int64_t Dk, int64_t Dv) {
    return N * H * ((Dv + ROWS - 1) / ROWS);
}

hipError_t launch_la_step(const LaStepArgs& a) {
    const int nb = (int)((a.Dv + ROWS - 1) / ROWS);
    const dim3 grid((unsigned)la_step_workgroups(a.N, a.H, a.Dk, a.Dv));
    auto go = [&](void (*kernel)(LaStepArgs, int)) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, a.stream, a, nb);
    };
    if (a.Dk <= 64) go(a.bf16 ? la_step_kernel<16, true> : la_step_kernel<16, false>);
    else go(a.bf16 ? la_step_kernel<32, true> : la_step_kernel<32, false>);
    return hipGetLastError();
}

}  // namespace gdr
