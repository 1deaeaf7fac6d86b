// combine_residual.cu -- the end of moe_layer: the routing-weighted top-k sum
// of the experts' rows (as combine.cu), normed, gated and scaled into the
// residual stream, and the next block's norm, in one pass.
//
//   y[t, m] = sum_{j = 0..k-1} w[t, j] * (y_sorted[2 r, m] + y_sorted[2 r + 1, m]),  r = inv[t*k + j]
//                                                              (paired rows; fp32, kept unrounded)
//   h'      = h + s * g * (y * r(y) * w_post),  x_next = h' * r(h') * w_next
//
// A token's row goes over a cluster of eight CTAs: at one token a single SM
// would have to pull all k rows (688 KB in 4 K parts at k=6, H=7168) through
// its own L2 port. The two row sums meet through distributed shared memory;
// each thread keeps its columns of y and h' in registers between them.
#include <cuda_bf16.h>

#include "moe_internal.h"
#include "ptx.cuh"
#include "row_ops.cuh"

namespace moe {

namespace {

constexpr int kClusterCtas = 8;
constexpr int kTailThreads = 256;
constexpr int kTailVecs = 2;      // float4 columns per thread: H <= 8 * 256 * 2 * 4 = 16384

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Sum of v over the cluster's threads, the same bits in every CTA: per warp,
// per CTA in warp order, then over the CTAs in rank order. slot: this sum's own shared word.
__device__ __forceinline__ float cluster_sum(float v, float *s_warp, float *slot)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0)
        s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        float c = 0.f;
        for (int i = 0; i < kTailThreads / 32; ++i)
            c += s_warp[i];
        *slot = c;
    }
    cluster_sync();
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < kClusterCtas; ++i)
        total += ld_cluster_f32(map_to_cta(smem_u32(slot), i));
    return total;
}

// kParts: K parts of y, part_stride elements apart, summed in part order as in
// combine.cu, each part's pair of rows first.
template <int kParts>
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kTailThreads, kParts == 1 ? 2 : 1)
    combine_residual_kernel(const float *y_sorted, const int32_t *inv, const float *w, const __grid_constant__ NormArgs a,
                            int k, size_t part_stride)
{
    __shared__ float s_warp[2][kTailThreads / 32];
    __shared__ float s_slot[2];
    const int t = blockIdx.x / kClusterCtas;
    const int cols = a.H / kClusterCtas;             // a multiple of 8
    const int m0 = static_cast<int>(cluster_ctarank()) * cols;
    // Ahead of the wait for y: the routing, h, the weights and the gate are
    // inputs of the call or were written two launches back or more, which is
    // complete (see launch_k), and of a token past the count nothing is used.
    constexpr int kRows = kParts == 2 ? 8 : 4;       // routed rows in flight
    constexpr int kSums = 2 * kParts;                // what a routed row is the sum of: its pair's parts
    int row[kRows];
    float wj[kRows];
    auto routing = [&](int j0) {
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            row[q] = j0 + q < k ? inv[t * k + j0 + q] : -1;
            wj[q] = j0 + q < k ? w[t * k + j0 + q] : 0.f;
        }
    };
    routing(0);
    float h[kTailVecs][4], wp[kTailVecs][4], wn[kTailVecs][4], g[kTailVecs][4];
#pragma unroll
    for (int v = 0; v < kTailVecs; ++v) {
        const int c = 4 * (threadIdx.x + v * kTailThreads);
        if (c >= cols)
            continue;
        const int m = m0 + c;
        load4(a.h, a.h_f32, t * a.h_stride + m, h[v]);
        weight4(a, a.norm_block ? a.w_post : nullptr, m, wp[v]);
        weight4(a, a.x ? a.w_next : nullptr, m, wn[v]);
        gate4(a, t, m, g[v]);
    }
    pdl_wait();
    pdl_trigger();
    int T = a.T_max;
    if (a.d_num_tokens) {
        T = *a.d_num_tokens;
        T = T < 0 ? 0 : (T > a.T_max ? a.T_max : T);
    }
    if (t >= T)      // the whole cluster
        return;
    float y[kTailVecs][4];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kTailVecs; ++v)
        y[v][0] = y[v][1] = y[v][2] = y[v][3] = 0.f;
    for (int j0 = 0; j0 < k; j0 += kRows) {
        if (j0 > 0)
            routing(j0);
#pragma unroll
        for (int v = 0; v < kTailVecs; ++v) {
            const int c = 4 * (threadIdx.x + v * kTailThreads);
            if (c >= cols)
                continue;
            float f[kRows][kSums][4];
#pragma unroll
            for (int q = 0; q < kRows; ++q)
#pragma unroll
                for (int p = 0; p < kSums; ++p)
                    if (row[q] >= 0) {
                        const float4 u = *reinterpret_cast<const float4 *>(
                            y_sorted + (p >> 1) * part_stride + (2 * static_cast<size_t>(row[q]) + (p & 1)) * a.H + m0 +
                            c);
                        f[q][p][0] = u.x; f[q][p][1] = u.y; f[q][p][2] = u.z; f[q][p][3] = u.w;
                    }
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                if (row[q] < 0)
                    continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float s = f[q][0][i];
#pragma unroll
                    for (int p = 1; p < kSums; ++p)
                        s = __fadd_rn(s, f[q][p][i]);
                    y[v][i] = __fadd_rn(y[v][i], __fmul_rn(wj[q], s));
                }
            }
        }
    }
#pragma unroll
    for (int v = 0; v < kTailVecs; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sum = fmaf(y[v][i], y[v][i], sum);
    const float r_y = a.norm_block ? 1.f / sqrtf(cluster_sum(sum, s_warp[0], &s_slot[0]) / a.H + a.eps) : 1.f;
    sum = 0.f;
#pragma unroll
    for (int v = 0; v < kTailVecs; ++v) {
        const int c = 4 * (threadIdx.x + v * kTailThreads);
        if (c >= cols)
            continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[v][i] = h[v][i] + a.scale * g[v][i] * (y[v][i] * r_y * wp[v][i]);
            sum = fmaf(y[v][i], y[v][i], sum);
        }
        const size_t o = t * a.out_stride + m0 + c;
        store4(a.h_out, a.h_f32, o, y[v]);
    }
    if (a.x) {
        const float r = 1.f / sqrtf(cluster_sum(sum, s_warp[1], &s_slot[1]) / a.H + a.eps);
#pragma unroll
        for (int v = 0; v < kTailVecs; ++v) {
            const int c = 4 * (threadIdx.x + v * kTailThreads);
            if (c >= cols)
                continue;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wn[v][i] = y[v][i] * r * wn[v][i];
            store4_bf16(a.x, t * a.x_stride + m0 + c, wn[v]);
        }
    }
    cluster_sync();   // no CTA leaves while another may still read its sums
}

}  // namespace

cudaError_t launch_combine_residual(const float *y_sorted, const int32_t *inv, const float *topk_weights,
                                    const NormArgs &a, int k, int parts, size_t part_stride, cudaStream_t stream,
                                    bool pdl)
{
    if (a.H > kClusterCtas * kTailThreads * kTailVecs * 4 || (parts != 1 && parts != 2 && parts != 4))
        return cudaErrorInvalidValue;
    auto kern = parts == 4 ? combine_residual_kernel<4> : (parts == 2 ? combine_residual_kernel<2> : combine_residual_kernel<1>);
    return launch_k(kern, dim3(static_cast<unsigned>(a.T_max) * kClusterCtas), dim3(kTailThreads), 0, stream, pdl,
                    y_sorted, inv, topk_weights, a, k, part_stride);
}

}  // namespace moe
