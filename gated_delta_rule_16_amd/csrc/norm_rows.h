// Rows that a wave or a workgroup holds in registers, 8 channels to an access: the
// reductions over them and the sum with the residual stream (layer norm, RMS norm).
#pragma once

#include "rows.h"

namespace gdr {

namespace {

constexpr int E = 8;              // channels per lane and access

constexpr int threads(int WR) { return WR == 8 ? 512 : 256; }

__device__ __forceinline__ float wave_sum(float x) {
    x += dpp_mov<0xB1>(x);
    x += dpp_mov<0x4E>(x);
    x += dpp_mov<0x141>(x);
    x += dpp_mov<0x140>(x);
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
    return x;
}

// A sum over WR waves of a row, in a fixed order.
template <int WR> __device__ __forceinline__ float join_waves(const float* red) {
    float x = (red[0] + red[1]) + (red[2] + red[3]);
    if constexpr (WR == 8) x += (red[4] + red[5]) + (red[6] + red[7]);
    return x;
}

// Sum over the row's threads: WR waves of a workgroup, or one wave.  `red`
// is one of alternating slots, so one barrier per sum suffices: a slot is
// written again only after the barrier of the sum in between.
template <int WR>
__device__ __forceinline__ float row_total(float x, float* red) {
    x = wave_sum(x);
    if constexpr (WR > 1) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = join_waves<WR>(red);
    }
    return x;
}

__device__ __forceinline__ int left(int64_t C, int64_t c) {
    const int64_t v = C - c;
    return v < 0 ? 0 : v > E ? E : (int)v;
}

// A thread's group of channels at c: how many it has (0 or E).  With RAG (C no
// multiple of E) the last group of the row is moved back to end with it; its
// first `twice` channels are those of the group before, and count there.
template <bool RAG>
__device__ __forceinline__ int own_group(int64_t& c, int64_t C, int& twice) {
    twice = 0;
    if (c >= C) return 0;
    if (RAG && c > C - E) {
        twice = (int)(c - (C - E));
        c = C - E;
    }
    return E;
}

// One group of channels of x (and r), and their sum h: rounded to the stored
// type, stored.  RES: 0 none, 1 bf16, 2 fp32.
template <bool BF16, int RES, bool RAG> struct SumIn {
    Row<E, BF16, RAG> x;
    Row<RES ? E : 1, RES == 1, RES ? RAG : false> r;
    template <class Args>
    __device__ __forceinline__ void load(const Args& a, int64_t row, int64_t c, int valid) {
        x.load(a.x, row * a.xr + c, valid);
        if constexpr (RES != 0) r.load(a.res, row * a.rr + c, valid);
    }
    __device__ __forceinline__ void sum(float (&h)[E]) {
        x.unpack(h);
        if constexpr (RES != 0) {
            float q[E];
            r.unpack(q);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                h[e] += q[e];
                if constexpr (RES == 1) h[e] = bf2f(f2bf(h[e]));
            }
        }
    }
};

}  // namespace

}  // namespace gdr
