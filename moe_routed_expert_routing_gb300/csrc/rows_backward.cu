// rows_backward.cu -- gradients of the rows' way into the sorted batch
// (dispatch) and back out of it (combine).
//
//   combine:   out[t] = sum_j w[t, j] y[inv[t, j]]
//     dy[inv[t, j]] = w[t, j] d_out[t],   dw[t, j] = <d_out[t], y[inv[t, j]]>
//   dispatch:  x_sorted[inv[t, j]] = x[t]
//     dx[t] = sum_j dx_sorted[inv[t, j]] (+ dx_add[t])
//
// Both go token by token, as the forward's combine does: every row of the
// sorted batch belongs to one slot, so each is read or written once, and the
// sums over a token's slots are a loop in ascending j: no atomics. Bound by HBM:
// T=8192, k=8, H=4096 combine 250 us for 1.68 GB (the copy rate), dispatch 93 us
// for 0.60 GB (0.97 of it). A few tokens: 2.6 us, the launch.
#include <cuda_bf16.h>

#include "moe_internal.h"
#include "tiles.cuh"

namespace moe {

namespace {

__device__ __forceinline__ int token_count(const int32_t *d_num_tokens, int T_max)
{
    if (!d_num_tokens)
        return T_max;
    const int T = *d_num_tokens;
    return T < 0 ? 0 : (T > T_max ? T_max : T);
}

// A row outside the batch counts as a dropped slot.
__device__ __forceinline__ int checked_row(int row, int cap) { return row < cap ? row : -1; }

__device__ __forceinline__ uint4 ld_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void widen8(const uint4 &u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

constexpr int kCombineThreads = 256;
constexpr int kRowsAtOnce = 4;

// One token per block: kRowsAtOnce of its slots at a time, their rows' loads
// issued together; a thread's products of each row are summed over the row's
// columns, then over the block.
template <bool kDot>
__global__ void __launch_bounds__(kCombineThreads) combine_backward_kernel(const uint4 *__restrict__ d_out,
                                                                           const float *__restrict__ y,
                                                                           const int32_t *__restrict__ inv,
                                                                           const float *__restrict__ w,
                                                                           const int32_t *d_num_tokens, int T_max,
                                                                           int k, int cap, int vec, uint4 *__restrict__ dy,
                                                                           float *__restrict__ dw)
{
    __shared__ float s_sum[kCombineThreads / 32][kRowsAtOnce];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int T = token_count(d_num_tokens, T_max);
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        const size_t slot0 = static_cast<size_t>(t) * k;
        for (int j0 = 0; j0 < k; j0 += kRowsAtOnce) {
            int row[kRowsAtOnce];
            float wj[kRowsAtOnce], sum[kRowsAtOnce];
#pragma unroll
            for (int q = 0; q < kRowsAtOnce; ++q) {
                const bool on = j0 + q < k;
                row[q] = on ? checked_row(__ldg(inv + slot0 + j0 + q), cap) : -1;
                wj[q] = on ? __ldg(w + slot0 + j0 + q) : 0.f;
                sum[q] = 0.f;
            }
            for (int c = threadIdx.x; c < vec; c += kCombineThreads) {
                const uint4 raw = __ldg(d_out + static_cast<size_t>(t) * vec + c);
                uint4 a[kRowsAtOnce], b[kRowsAtOnce];
                if constexpr (kDot) {
#pragma unroll
                    for (int q = 0; q < kRowsAtOnce; ++q)
                        if (row[q] >= 0) {
                            const float *p = y + (static_cast<size_t>(row[q]) * vec + c) * 8;
                            a[q] = ld_stream(p);
                            b[q] = ld_stream(p + 4);
                        }
                }
                float d[8];
                widen8(raw, d);
#pragma unroll
                for (int q = 0; q < kRowsAtOnce; ++q) {
                    if (row[q] < 0)
                        continue;
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[i] = wj[q] * d[i];
                    dy[static_cast<size_t>(row[q]) * vec + c] = narrow8(o);
                    if constexpr (kDot) {
                        const uint32_t u[8] = {a[q].x, a[q].y, a[q].z, a[q].w, b[q].x, b[q].y, b[q].z, b[q].w};
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sum[q] = fmaf(d[i], __uint_as_float(u[i]), sum[q]);
                    }
                }
            }
            if constexpr (kDot) {
#pragma unroll
                for (int q = 0; q < kRowsAtOnce; ++q) {
#pragma unroll
                    for (int o = 16; o; o >>= 1)
                        sum[q] += __shfl_xor_sync(kFull, sum[q], o);
                    if (lane == 0)
                        s_sum[warp][q] = sum[q];
                }
                __syncthreads();
                if (threadIdx.x < kRowsAtOnce && j0 + static_cast<int>(threadIdx.x) < k) {
                    float v = 0.f;
#pragma unroll
                    for (int i = 0; i < kCombineThreads / 32; ++i)
                        v += s_sum[i][threadIdx.x];
                    dw[slot0 + j0 + threadIdx.x] = v;   // a dropped slot's sum is 0
                }
                __syncthreads();
            }
        }
    }
}

constexpr int kDispatchBwdThreads = 128;
constexpr long long kGridPerSm = 8;

// One item = one token x 1024 columns. The rows of eight slots (fp32: four) are
// loaded together, and while they are on their way the next item's first slots
// are read, so that no trip for the routing stands between one item's rows and
// the next's (T=1021, k=6, H=7168 with inputs from HBM 22.9 -> 20.7 us).
template <bool kF32>
__global__ void __launch_bounds__(kDispatchBwdThreads, 8) dispatch_backward_kernel(const void *__restrict__ dx_sorted,
                                                                                   const int32_t *__restrict__ inv,
                                                                                   const uint4 *add,
                                                                                   const int32_t *d_num_tokens,
                                                                                   int T_max, int k, int cap, int vec,
                                                                                   uint4 *dx)
{
    constexpr int kRows = kF32 ? 4 : 8;
    const int groups = (vec + kDispatchBwdThreads - 1) / kDispatchBwdThreads;
    const long long items = static_cast<long long>(token_count(d_num_tokens, T_max)) * groups;
    int next[kRows];
    auto slots = [&](long long item, int j0) {
        const int32_t *inv_t = inv + item / groups * k;
#pragma unroll
        for (int q = 0; q < kRows; ++q)
            next[q] = item < items && j0 + q < k ? checked_row(__ldg(inv_t + j0 + q), cap) : -1;
    };
    slots(blockIdx.x, 0);
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const int t = static_cast<int>(item / groups);
        const int c = static_cast<int>(item - static_cast<long long>(t) * groups) * kDispatchBwdThreads + threadIdx.x;
        const bool mine = c < vec;
        const size_t at = static_cast<size_t>(t) * vec + c;
        uint4 more = make_uint4(0u, 0u, 0u, 0u);
        if (add && mine)
            more = ld_stream(add + at);
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < k; j0 += kRows) {
            uint4 a[kRows], b[kF32 ? kRows : 1];
            unsigned on = 0;
#pragma unroll
            for (int q = 0; q < kRows; ++q)
                if (mine && next[q] >= 0) {
                    on |= 1u << q;
                    const size_t i = static_cast<size_t>(next[q]) * vec + c;
                    if constexpr (kF32) {
                        a[q] = ld_stream(static_cast<const float *>(dx_sorted) + i * 8);
                        b[q] = ld_stream(static_cast<const float *>(dx_sorted) + i * 8 + 4);
                    } else {
                        a[q] = ld_stream(static_cast<const uint4 *>(dx_sorted) + i);
                    }
                }
            if (j0 + kRows < k)
                slots(item, j0 + kRows);
            else
                slots(item + gridDim.x, 0);
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                if (!(on >> q & 1u))
                    continue;
                float f[8];
                if constexpr (kF32) {
                    const uint32_t u[8] = {a[q].x, a[q].y, a[q].z, a[q].w, b[q].x, b[q].y, b[q].z, b[q].w};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        f[i] = __uint_as_float(u[i]);
                } else {
                    widen8(a[q], f);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] += f[i];
            }
        }
        if (!mine)
            continue;
        if (add) {
            float f[8];
            widen8(more, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i] += f[i];
        }
        dx[at] = narrow8(acc);
    }
}

}  // namespace

cudaError_t launch_combine_backward(const void *d_out, const float *y_sorted, const int32_t *inv,
                                    const float *topk_weights, const int32_t *d_num_tokens, int T_max, int k, int cap,
                                    int H, void *dy_sorted, float *d_weights, int num_sms, cudaStream_t stream)
{
    const int most = num_sms * 8;
    const dim3 grid(T_max < most ? T_max : most);
    auto kern = d_weights ? combine_backward_kernel<true> : combine_backward_kernel<false>;
    return launch_k(kern, grid, dim3(kCombineThreads), 0, stream, false, static_cast<const uint4 *>(d_out), y_sorted,
                    inv, topk_weights, d_num_tokens, T_max, k, cap, H / 8, static_cast<uint4 *>(dy_sorted), d_weights);
}

cudaError_t launch_dispatch_backward(const void *dx_sorted, bool f32, const int32_t *inv, const void *dx_add,
                                     const int32_t *d_num_tokens, int T_max, int k, int cap, int H, void *dx, int num_sms,
                                     cudaStream_t stream)
{
    const int vec = H / 8;
    const long long items = static_cast<long long>(T_max) * ((vec + kDispatchBwdThreads - 1) / kDispatchBwdThreads);
    const long long most = num_sms * kGridPerSm;
    const dim3 grid(static_cast<unsigned>(items < most ? items : most));
    auto kern = f32 ? dispatch_backward_kernel<true> : dispatch_backward_kernel<false>;
    return launch_k(kern, grid, dim3(kDispatchBwdThreads), 0, stream, false, dx_sorted, inv,
                    static_cast<const uint4 *>(dx_add), d_num_tokens, T_max, k, cap, vec, static_cast<uint4 *>(dx));
}

}  // namespace moe
