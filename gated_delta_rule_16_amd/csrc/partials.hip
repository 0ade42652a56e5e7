// Sums of the workgroups' partial gradients of parameters (convolution, layer
// norm), in a fixed order, so results do not vary from run to run.
#include "block_launch.h"
#include "rows.h"

namespace gdr {

namespace {

// out[m] = sum over p of part[p][m], one lane per m: a workgroup owns 64
// columns, each of its W waves every W-th p (8 loads in flight), joined through
// LDS.  The first m0 columns go to o0, the others to o1 (either may be NULL).
template <int W>
__global__ __launch_bounds__(64 * W) void sum_partials_kernel(const float* __restrict__ part,
                                                              int64_t P, int64_t M, float* o0,
                                                              int64_t m0, float* o1) {
    __shared__ float red[W][64];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m = (int64_t)blockIdx.x * 64 + lane;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (m < M) {
        int64_t p = wv;
        for (; p + 7 * W < P; p += 8 * W)
#pragma unroll
            for (int u = 0; u < 8; ++u) s[u] += part[(p + u * W) * M + m];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (p + u * W < P) s[u] += part[(p + u * W) * M + m];
    }
    red[wv][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    if (wv == 0 && m < M) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < W; w += 4)
            v += (red[w][lane] + red[w + 1][lane]) + (red[w + 2][lane] + red[w + 3][lane]);
        if (m < m0) {
            if (o0) o0[m] = v;
        } else if (o1) {
            o1[m - m0] = v;
        }
    }
}

}  // namespace

hipError_t launch_sum_partials(const float* part, int64_t P, int64_t M, float* o0, int64_t m0,
                               float* o1, hipStream_t st) {
    const dim3 grid((unsigned)((M + 63) / 64));
    // many rows: 16 waves a workgroup (1024 rows of 4096: 17 -> 6 us)
    if (P >= 64)
        hipLaunchKernelGGL((sum_partials_kernel<16>), grid, dim3(1024), 0, st, part, P, M, o0, m0,
                           o1);
    else
        hipLaunchKernelGGL((sum_partials_kernel<4>), grid, dim3(256), 0, st, part, P, M, o0, m0,
                           o1);
    return hipGetLastError();
}

}  // namespace gdr
