// route.cu -- the router: logits of every expert, scores, and the k experts
// of the largest keys with their weights.
#include <cuda_bf16.h>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int token_count(const int32_t *d_num_tokens, int T_max)
{
    int T = T_max;
    if (d_num_tokens) {
        T = *d_num_tokens;
        T = T < 0 ? 0 : (T > T_max ? T_max : T);
    }
    return T;
}

// logits[t, e] = sum_m x[t, m] w[e, m]: 64 x 64 tiles, 16-wide K steps, 4 x 4 per thread.
__global__ void __launch_bounds__(256) logits_kernel(const RouteArgs a)
{
    __shared__ float sx[16][65], sw[16][65];
    const int T = token_count(a.d_num_tokens, a.T_max);
    const int t0 = blockIdx.x * 64, e0 = blockIdx.y * 64;
    if (t0 >= T)
        return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int m0 = 0; m0 < a.H; m0 += 16) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i >> 4, c = i & 15;
            const size_t xi = static_cast<size_t>(t0 + r) * a.H + m0 + c;
            float v = 0.f;
            if (t0 + r < T)
                v = a.x_f32 ? static_cast<const float *>(a.x)[xi]
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.x)[xi]);
            sx[c][r] = v;
            sw[c][r] = e0 + r < a.E ? __bfloat162float(static_cast<const __nv_bfloat16 *>(
                                          a.w)[static_cast<size_t>(e0 + r) * a.H + m0 + c])
                                    : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] += sx[c][ty * 4 + i] * sw[c][tx * 4 + j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (t0 + ty * 4 + i < T && e0 + tx * 4 + j < a.E)
                a.logits[static_cast<size_t>(t0 + ty * 4 + i) * a.E + e0 + tx * 4 + j] = acc[i][j];
}

// A float as an unsigned integer of the same order; 0 for what may not be
// chosen (-inf and NaN). -0 and +0 give the same number.
__device__ __forceinline__ uint32_t order_key(float f)
{
    f = f + 0.f;
    const uint32_t b = __float_as_uint(f);
    const uint32_t u = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return f > -INFINITY ? u : 0u;   // false for NaN too
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// log of the sigmoid, without overflow or a loss of small values
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.f) - log1pf(expf(-fabsf(l))); }

// One warp selects for one token: lane i holds the logits of experts i, i + 32, ...
// s_key[E]: this warp's scratch, used with groups only.
template <int kPer>
__device__ void select_experts(const RouteArgs &a, int t, float (&l)[kPer], float *s_key)
{
    const int lane = threadIdx.x & 31;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool real = lane + 32 * i < a.E;
        if (real && !(l[i] < INFINITY)) {   // NaN or +inf
            bad = true;
            l[i] = -INFINITY;
        }
        if (!real)
            l[i] = -INFINITY;
    }
    if (__any_sync(kFull, bad) && lane == 0)
        atomicOr(a.err, MOE_DEVERR_BAD_LOGIT);
    float mx = -INFINITY, sum = 1.f;
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            mx = fmaxf(mx, l[i]);
        mx = warp_max(mx);
        mx = mx > -INFINITY ? mx : 0.f;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            sum += expf(l[i] - mx);
        sum = warp_sum(sum);
    }
    auto score = [&](float v) { return a.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - mx) / sum; };
    const bool by_score = a.bias != nullptr || a.group_top > 1;
    uint32_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        float v = l[i];
        if (by_score && e < a.E && v > -INFINITY)
            v = score(v) + (a.bias ? a.bias[e] : 0.f);
        key[i] = e < a.E ? order_key(v) : 0u;
        if (a.n_group > 1 && e < a.E)
            s_key[e] = key[i] ? v : -INFINITY;
    }
    if (a.n_group > 1) {
        __syncwarp();
        const int gs = a.E / a.n_group;
        float value = -INFINITY;
        if (lane < a.n_group) {
            float first = -INFINITY, second = -INFINITY;
            for (int i = 0; i < gs; ++i) {
                const float v = s_key[lane * gs + i];
                if (v > first) {
                    second = first;
                    first = v;
                } else if (v > second) {
                    second = v;
                }
            }
            value = a.group_top > 1 ? first + second : first;
            if (!(value > -INFINITY))   // also inf - inf
                value = -INFINITY;
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const float o = __shfl_sync(kFull, value, g);
            rank += (o > value || (o == value && g < lane)) ? 1 : 0;
        }
        const unsigned kept = __ballot_sync(kFull, lane < a.n_group && rank < a.topk_group);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((kept >> (e / gs)) & 1u))
                key[i] = 0u;
        }
        __syncwarp();
    }
    // k rounds: the largest key, the lowest expert among equals
    int my_id[2] = {-1, -1};       // lane j holds places j and j + 32
    float my_l[2] = {-INFINITY, -INFINITY};
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
        int at = 1 << 30;
        float val = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
                val = l[i];
            }
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == 0u)
            break;
        const int e = __reduce_min_sync(kFull, best == top ? at : 1 << 30);
        val = __shfl_sync(kFull, val, e & 31);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i == e)
                key[i] = 0u;
        if (lane == (j & 31)) {
            my_id[j >> 5] = e;
            my_l[j >> 5] = val;
        }
    }
    // weights
    float w[2], norm = 1.f;
    if (a.renormalize) {
        // the chosen scores over their sum, from their logarithms (the softmax
        // over all E cancels), so that scores that underflow keep their ratios
        float lg[2], m2 = -INFINITY;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            lg[q] = my_id[q] >= 0 ? (a.sigmoid ? log_sigmoid(my_l[q]) : my_l[q]) : -INFINITY;
            m2 = fmaxf(m2, lg[q]);
        }
        m2 = warp_max(m2);
        m2 = m2 > -INFINITY ? m2 : 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w[q] = expf(lg[q] - m2);
        norm = warp_sum(w[0] + w[1]);
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w[q] = my_id[q] >= 0 ? score(my_l[q]) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = lane + 32 * q;
        if (j < a.k) {
            a.ids[static_cast<size_t>(t) * a.k + j] = my_id[q];
            a.weights[static_cast<size_t>(t) * a.k + j] = my_id[q] >= 0 ? a.scale * (w[q] / norm) : 0.f;
        }
    }
}

constexpr int kSelectWarps = 4;

template <int kPer>
__global__ void __launch_bounds__(32 * kSelectWarps) select_kernel(const RouteArgs a)
{
    __shared__ float s_key[kSelectWarps][kPer * 32];
    const int T = token_count(a.d_num_tokens, a.T_max);
    const int t = blockIdx.x * kSelectWarps + (threadIdx.x >> 5);
    if (t >= T)
        return;
    const int lane = threadIdx.x & 31;
    float l[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        l[i] = lane + 32 * i < a.E ? a.logits[static_cast<size_t>(t) * a.E + lane + 32 * i] : 0.f;
    select_experts<kPer>(a, t, l, s_key[threadIdx.x >> 5]);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, int num_sms, cudaStream_t stream, bool pdl)
{
    (void)num_sms;
    (void)pdl;
    cudaError_t e = launch_k(logits_kernel, dim3((a.T_max + 63) / 64, (a.E + 63) / 64), dim3(256), 0, stream, false, a);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((a.T_max + kSelectWarps - 1) / kSelectWarps), block(32 * kSelectWarps);
    if (a.E <= 128)
        return launch_k(select_kernel<4>, grid, block, 0, stream, false, a);
    if (a.E <= 256)
        return launch_k(select_kernel<8>, grid, block, 0, stream, false, a);
    if (a.E <= 512)
        return launch_k(select_kernel<16>, grid, block, 0, stream, false, a);
    return launch_k(select_kernel<32>, grid, block, 0, stream, false, a);
}

}  // namespace moe
