// Sums of per-workgroup partial gradients, and of the scan's per-block B and
// C gradients.  Every sum runs in a fixed order, so results do not vary from
// run to run.
#include "launch.h"
#include "rows.h"

namespace gdr {

namespace {

// out[m] = sum over p of part[p][m], one lane per m: a workgroup owns 64
// columns, each of its four waves every fourth p, joined through LDS.  The
// columns are cut into up to three outputs.
__global__ __launch_bounds__(256) void sum_partials_kernel(const float* __restrict__ part,
                                                           int64_t P, int64_t M, float* o0,
                                                           int64_t m0, float* o1, int64_t m1,
                                                           float* o2) {
    __shared__ float red[4][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 64 + lane;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (m < M) {
        int64_t p = wv;
        for (; p + 12 < P; p += 16)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] += part[(p + 4 * u) * M + m];
        for (; p < P; p += 4) s[0] += part[p * M + m];
    }
    red[wv][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (wv == 0 && m < M) {
        const float v = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
        if (m < m0) {
            if (o0) o0[m] = v;
        } else if (m < m0 + m1) {
            if (o1) o1[m - m0] = v;
        } else if (o2) {
            o2[m - m0 - m1] = v;
        }
    }
}

}  // namespace

hipError_t launch_sum_partials(const float* part, int64_t P, int64_t M, float* o0, int64_t m0,
                               float* o1, int64_t m1, float* o2, hipStream_t st) {
    hipLaunchKernelGGL(sum_partials_kernel, dim3((unsigned)((M + 63) / 64)), dim3(256), 0, st,
                       part, P, M, o0, m0, o1, m1, o2);
    return hipGetLastError();
}

}  // namespace gdr
