// Pieces shared by the selective scan's kernels (forward, backward, token).
//
// Lane layout of every scan kernel: a lane holds 4 neighbouring states of one
// channel; LPC = 1, 2, 4, 8 or 16 neighbouring lanes share the channel (N up
// to 4 LPC states), so a wave runs 64 / LPC channels and a workgroup of four
// waves WC = 256 / LPC.  States n >= N of the last lane have A = B = C = 0 and
// stay 0.
#pragma once

#include "launch.h"
#include "rows.h"

namespace gdr {

// Value of lane l ^ M (M = 1, 2, 4, 8): DPP moves, no LDS traffic.
template <int M>
__device__ __forceinline__ float xor_lane(float x) {
    const int i = __builtin_bit_cast(int, x);
    if constexpr (M == 1) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, i, 0xB1, 0xF, 0xF, false));
    if constexpr (M == 2) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, i, 0x4E, 0xF, 0xF, false));
    if constexpr (M == 8) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, i, 0x128, 0xF, 0xF, false));
    static_assert(M == 1 || M == 2 || M == 4 || M == 8, "lane distance");
    // banks 0 and 2 of a row read 4 lanes up (row_shl 4), banks 1 and 3 down
    const int up = __builtin_amdgcn_update_dpp(0, i, 0x104, 0xF, 0x5, false);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(up, i, 0x114, 0xF, 0xA, false));
}

// One step of a halving reduction: lanes with bit M clear keep a's sum of the
// pair (l, l ^ M), lanes with it set b's.
template <int M>
__device__ __forceinline__ float fold(float a, float b, bool bit) {
    return (bit ? b : a) + xor_lane<M>(bit ? a : b);
}

// The same across 16 or 32 lanes, one swap and one add.
__device__ __forceinline__ float fold16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a),
                                                    __builtin_bit_cast(unsigned, b), false, false);
    return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}
__device__ __forceinline__ float fold32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a),
                                                    __builtin_bit_cast(unsigned, b), false, false);
    return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}

// Sums s[k] (token k of 4) over the LPC lanes of each channel and stores them
// at dst[k * pitch]; each lane stores what the halving left it, so a group of
// 4 tokens costs few stores.  li = lane % LPC.
template <int LPC>
__device__ __forceinline__ void channel_sums(const float (&s)[4], int li, float* dst, int pitch) {
    if constexpr (LPC == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k * pitch] = s[k];
    } else {
        const bool b0 = li & 1;
        const float p0 = fold<1>(s[0], s[1], b0), p1 = fold<1>(s[2], s[3], b0);
        if constexpr (LPC == 2) {
            dst[(li & 1) * pitch] = p0;
            dst[(2 + (li & 1)) * pitch] = p1;
        } else {
            float r = fold<2>(p0, p1, li & 2);
            if constexpr (LPC >= 8) r += xor_lane<4>(r);
            if constexpr (LPC >= 16) r += xor_lane<8>(r);
            if (LPC == 4 || li < 4) dst[(li & 3) * pitch] = r;
        }
    }
}

// Four states of one lane in memory ([.., N] floats, element-aligned).
__device__ __forceinline__ void state_load(float (&h)[4], const float* p, int valid) {
    param_load<4>(h, p, valid);
}
__device__ __forceinline__ void state_store(float* p, const float (&h)[4], int valid) {
    row_store<4>(p, 0, false, h, valid);
}

// The step Delta of a token and channel.
__device__ __forceinline__ float ssm_delta(float raw, bool sp) { return sp ? softplus(raw) : raw; }

// Valid states of a lane.
__device__ __forceinline__ int ssm_states(int64_t N, int ng) {
    const int64_t v = N - 4 * ng;
    return v < 0 ? 0 : v > 4 ? 4 : (int)v;
}

__device__ __forceinline__ int ssm_left(int64_t lim, int64_t c, int e) {
    const int64_t v = lim - c;
    return v < 0 ? 0 : v > e ? e : (int)v;
}

}  // namespace gdr
