// norm_ops.cuh -- a thread's columns of a residual row in packed pairs of fp32,
// and sums over the threads of a row (norm.cu, norm_backward.cu).
#pragma once

#include <type_traits>

#include <cuda_bf16.h>

#include "moe_internal.h"

namespace moe {

namespace {

__device__ __forceinline__ uint4 ld_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint2 ld_stream2(const void *p)
{
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// ---- packed pairs of fp32 ----

using Pair = unsigned long long;

__device__ __forceinline__ Pair pair(float lo, float hi)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}

__device__ __forceinline__ float2 halves(Pair p)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}

__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ Pair widen(uint32_t u)   // two bf16
{
    return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

__device__ __forceinline__ uint32_t narrow(Pair p)
{
    const float2 f = halves(p);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// A thread's unit is 16 bytes of the residual stream: 8 columns of bf16 or 4 of fp32.
template <bool kF32>
struct Unit {
    static constexpr int kCols = kF32 ? 4 : 8;
    static constexpr int kPairs = kCols / 2;
    using Half = typename std::conditional<kF32, uint2, uint4>::type;   // the same columns in bf16

    static __device__ __forceinline__ Half load_half(const __nv_bfloat16 *p)
    {
        if constexpr (kF32)
            return ld_stream2(p);
        else
            return ld_stream(p);
    }

    static __device__ __forceinline__ void pairs(const uint4 &u, Pair (&f)[kPairs])
    {
        if constexpr (kF32) {
            f[0] = pair(__uint_as_float(u.x), __uint_as_float(u.y));
            f[1] = pair(__uint_as_float(u.z), __uint_as_float(u.w));
        } else {
            f[0] = widen(u.x); f[1] = widen(u.y); f[2] = widen(u.z); f[3] = widen(u.w);
        }
    }

    static __device__ __forceinline__ void half_pairs(const Half &u, Pair (&f)[kPairs])
    {
        f[0] = widen(u.x);
        f[1] = widen(u.y);
        if constexpr (!kF32) {
            f[2] = widen(u.z);
            f[3] = widen(u.w);
        }
    }

    static __device__ __forceinline__ void store_half(__nv_bfloat16 *p, const Pair (&f)[kPairs])
    {
        if constexpr (kF32)
            *reinterpret_cast<uint2 *>(p) = make_uint2(narrow(f[0]), narrow(f[1]));
        else
            *reinterpret_cast<uint4 *>(p) = make_uint4(narrow(f[0]), narrow(f[1]), narrow(f[2]), narrow(f[3]));
    }

    static __device__ __forceinline__ void store(void *p, const Pair (&f)[kPairs])
    {
        if constexpr (kF32) {
            const float2 a = halves(f[0]), b = halves(f[1]);
            *static_cast<float4 *>(p) = make_float4(a.x, a.y, b.x, b.y);
        } else {
            store_half(static_cast<__nv_bfloat16 *>(p), f);
        }
    }

    // kCols values of a per-channel vector of either type
    static __device__ __forceinline__ void channel(const void *p, bool f32, int m, Pair (&f)[kPairs])
    {
        if (f32) {
#pragma unroll
            for (int i = 0; i < kPairs; i += 2) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + m + 2 * i));
                f[i] = pair(v.x, v.y);
                f[i + 1] = pair(v.z, v.w);
            }
        } else {
            half_pairs(__ldg(reinterpret_cast<const Half *>(static_cast<const __nv_bfloat16 *>(p) + m)), f);
        }
    }

    // c *= the norm weight w' of the columns from m on (w null: 1)
    static __device__ __forceinline__ void times_weight(const NormArgs &a, const void *w, int m, Pair (&c)[kPairs])
    {
        if (!w)
            return;
        Pair v[kPairs];
        channel(w, a.w_f32, m, v);
        if (a.unit_offset) {
            const Pair one = pair(1.f, 1.f);
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                v[i] = add2(v[i], one);
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            c[i] = mul2(c[i], v[i]);
    }
};

// Sum over the tpr threads of a row group (whole warps); every thread of the
// block calls it. s: this sum's words, one per warp of the block.
__device__ __forceinline__ float row_sum(Pair q, int tpr, float *s)
{
    const float2 f = halves(q);
    float v = f.x + f.y;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32)
        return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        s[warp] = v;
    __syncthreads();
    const int n = tpr >> 5;      // at most 16
    v = lane < n ? s[warp / n * n + lane] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
}

}  // namespace

}  // namespace moe
