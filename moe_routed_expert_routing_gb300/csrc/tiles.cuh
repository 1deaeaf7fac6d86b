// tiles.cuh -- row tiles of a batch sorted by expert, as every CTA of the
// grouped GEMMs finds them from the device-resident offsets (grouped_gemm.cu,
// expert_backward.cu).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace moe {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// Largest e in [0, E) with tp[e] * scale <= u (tp non-decreasing, tp[0] = 0).
__device__ __forceinline__ int find_expert(const int *tp, int E, int u, int scale)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tp[mid] * scale <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Per-expert row-tile prefix (one warp): s_tp[e] = sum_{e' < e} ceil(rows(e') / tile_rows).
__device__ __forceinline__ void build_tile_prefix(const int *s_off, int *s_tp, int E, int tile_rows, int lane)
{
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
        const int e = base + lane;
        int tiles = 0;
        if (e < E) {
            int c = s_off[e + 1] - s_off[e];
            c = c < 0 ? 0 : c;
            tiles = (c + tile_rows - 1) / tile_rows;
        }
        int v = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(kFull, v, o);
            if (lane >= o)
                v += n;
        }
        if (e < E)
            s_tp[e] = carry + v - tiles;
        carry += __shfl_sync(kFull, v, 31);
    }
    if (lane == 0)
        s_tp[E] = carry;
}

}  // namespace

}  // namespace moe
