// row_ops.cuh -- four columns of a residual row, a norm weight or a gate, in
// fp32 (the ends of moe_layer: combine_residual.cu, grouped_gemm.cu).
#pragma once

#include <cuda_bf16.h>

#include "moe_internal.h"

namespace moe {

namespace {

__device__ __forceinline__ void load4(const void *p, bool f32, size_t i, float (&f)[4])
{
    if (f32) {
        const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i);
        f[0] = __uint_as_float(v.x << 16);
        f[1] = __uint_as_float(v.x & 0xffff0000u);
        f[2] = __uint_as_float(v.y << 16);
        f[3] = __uint_as_float(v.y & 0xffff0000u);
    }
}

__device__ __forceinline__ void store4_bf16(void *p, size_t i, const float (&f)[4])
{
    const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t *>(&lo);
    o.y = *reinterpret_cast<const uint32_t *>(&hi);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p) + i) = o;
}

__device__ __forceinline__ void weight4(const NormArgs &a, const void *w, int m, float (&f)[4])
{
    if (!w) {
        f[0] = f[1] = f[2] = f[3] = 1.f;
        return;
    }
    load4(w, a.w_f32, m, f);
    if (a.unit_offset)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = 1.f + f[i];
}

__device__ __forceinline__ void store4(void *p, bool f32, size_t i, const float (&f)[4])
{
    if (f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
    else
        store4_bf16(p, i, f);
}

// The gate of token t's columns m..m + 3
__device__ __forceinline__ void gate4(const NormArgs &a, int t, int m, float (&g)[4])
{
    g[0] = g[1] = g[2] = g[3] = 1.f;
    if (a.gate_kind == MOE_GATE_CHANNEL)
        load4(a.gate, a.w_f32, m, g);
    else if (a.gate_kind == MOE_GATE_TOKEN)
        g[0] = g[1] = g[2] = g[3] = static_cast<const float *>(a.gate)[t];
    else if (a.gate_kind == MOE_GATE_ELEMENT)
        load4(a.gate, false, t * a.gate_stride + m, g);
}

}  // namespace

}  // namespace moe
