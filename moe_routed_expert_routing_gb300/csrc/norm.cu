// norm.cu -- the norm of the residual stream before the block, and the way
// back into it after the block: norm of the block's output, gate, residual
// scale, and the next block's norm in the same pass.
//
//   moe_norm:           x = h * r(h) * w
//   moe_norm_residual:  h' = h + s * g * (y * r(y) * w_post),  x_next = h' * r(h') * w_next
//   r(v) = 1 / sqrt(mean(v^2) + eps)
//
// All sums and products in fp32, one rounding per output.
#include <cuda_bf16.h>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float load_f(const void *p, bool f32, size_t i)
{
    return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ float weight_at(const NormArgs &a, const void *w, int m)
{
    if (!w)
        return 1.f;
    const float v = load_f(w, a.w_f32, m);
    return a.unit_offset ? 1.f + v : v;
}

__device__ __forceinline__ float block_sum(float v)
{
    __shared__ float s[kNormThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kNormThreads / 32; ++i)
        v += s[i];
    return v;
}

__device__ __forceinline__ float gate_at(const NormArgs &a, int t, int m)
{
    switch (a.gate_kind) {
    case MOE_GATE_CHANNEL:
        return load_f(a.gate, a.w_f32, m);
    case MOE_GATE_TOKEN:
        return static_cast<const float *>(a.gate)[t];
    case MOE_GATE_ELEMENT:
        return load_f(a.gate, false, static_cast<size_t>(t) * a.gate_stride + m);
    default:
        return 1.f;
    }
}

__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormArgs a)
{
    extern __shared__ float row[];
    int T = a.T_max;
    if (a.d_num_tokens) {
        T = *a.d_num_tokens;
        T = T < 0 ? 0 : (T > a.T_max ? a.T_max : T);
    }
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        float r_y = 1.f;
        if (a.y && a.norm_block) {
            float q = 0.f;
            for (int m = threadIdx.x; m < a.H; m += kNormThreads) {
                const float v = load_f(a.y, false, static_cast<size_t>(t) * a.y_stride + m);
                q += v * v;
            }
            r_y = rsqrtf(block_sum(q) / a.H + a.eps);
        }
        float q = 0.f;
        for (int m = threadIdx.x; m < a.H; m += kNormThreads) {
            float v = load_f(a.h, a.h_f32, static_cast<size_t>(t) * a.h_stride + m);
            if (a.y) {
                float n = load_f(a.y, false, static_cast<size_t>(t) * a.y_stride + m);
                if (a.norm_block)
                    n = n * r_y * weight_at(a, a.w_post, m);
                v = v + a.scale * gate_at(a, t, m) * n;
                const size_t o = static_cast<size_t>(t) * a.out_stride + m;
                if (a.h_f32)
                    static_cast<float *>(a.h_out)[o] = v;
                else
                    static_cast<__nv_bfloat16 *>(a.h_out)[o] = __float2bfloat16_rn(v);
            }
            row[m] = v;
            q += v * v;
        }
        if (!a.x)
            continue;
        const float r = rsqrtf(block_sum(q) / a.H + a.eps);
        for (int m = threadIdx.x; m < a.H; m += kNormThreads)
            static_cast<__nv_bfloat16 *>(a.x)[static_cast<size_t>(t) * a.x_stride + m] =
                __float2bfloat16_rn(row[m] * r * weight_at(a, a.w_next, m));
    }
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t stream, bool pdl)
{
    const size_t smem = sizeof(float) * a.H;
    cudaError_t e = cudaFuncSetAttribute(norm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 32768 * 4);
    if (e != cudaSuccess)
        return e;
    const int grid = a.T_max < num_sms * 8 ? a.T_max : num_sms * 8;
    (void)pdl;
    return launch_k(norm_kernel, dim3(grid), dim3(kNormThreads), smem, stream, false, a);
}

}  // namespace moe
