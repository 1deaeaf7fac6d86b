// route_backward.cu -- the router's gradient up to its logits, and sums of
// partial products.
//
// The forward's weights are w_j = scale c_j, or scale c_j / S with S = sum_i c_i,
// of the chosen experts' scores c_j. With v_j = c_j / S:
//   softmax, renormalised: S cancels the softmax's sum, so v is the softmax of
//     the chosen logits alone: dl_j = scale v_j (dw_j - sum_i dw_i v_i), 0 elsewhere
//   softmax:  dl_e = p_e (scale [e chosen] dw_e - scale sum_i dw_i p_i), every e
//   sigmoid, renormalised: dl_j = scale v_j (1 - c_j) (dw_j - sum_i dw_i v_i)
//   sigmoid:  dl_j = scale dw_j c_j (1 - c_j)
// No gradient goes through the choice itself, nor to the selection bias. v of
// sigmoid scores is formed from their logarithms, so scores that underflow
// still have their ratio.
//
// dx = dl w_router and dw_router = dl^T x are products on the tensor cores
// (expert_backward.cu), which take bf16: dl goes to them as two bf16 parts,
// leading part and rest, so it counts with 16 bits, a relative 2^-16 off at
// most; both products' sums stay fp32. One part would cost a gradient 1.7e-3 of
// its rms, as much as a bf16 output's own rounding; a third part (24 bits) would
// show in an fp32 dw_router only.
#include <cuda_bf16.h>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A logit as the router takes it: NaN and +inf count as -inf.
__device__ __forceinline__ float as_logit(float l) { return l < INFINITY ? l : -INFINITY; }

// One warp per token. Its row of dl grows in shared memory: base values, then
// the chosen experts' terms, each added by the lane its expert falls to.
__global__ void __launch_bounds__(kThreads) route_grad_kernel(const __grid_constant__ RouteGradArgs a)
{
    extern __shared__ float4 s_row[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, k = a.k, Ep = (E + 63) & ~63;
    const bool whole = E % 4 == 0;
    float *const dl = reinterpret_cast<float *>(s_row) + warp * Ep;
    pdl_wait();
    pdl_trigger();
    int T = a.T_max;
    if (a.d_num_tokens) {
        T = *a.d_num_tokens;
        T = T < 0 ? 0 : (T > a.T_max ? a.T_max : T);
    }
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s <= a.segments; s += kThreads)
            a.offsets[s] = static_cast<int>(min(static_cast<long long>(T), static_cast<long long>(s) * a.segment_rows));
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < Ep; i += kThreads)     // 2 Ep bf16 zeros
            reinterpret_cast<uint32_t *>(a.parts)[static_cast<size_t>(a.T_max) * Ep + i] = 0u;
    for (int t = blockIdx.x * (kThreads / 32) + warp; t < T; t += gridDim.x * (kThreads / 32)) {
        const float *const logits = a.logits + static_cast<size_t>(t) * E;
        const int32_t *const ids = a.ids + static_cast<size_t>(t) * k;
        const float *const dw = a.d_weights + static_cast<size_t>(t) * k;
        // the chosen experts' logits and gradients: slots lane and lane + 32
        int id[2];
        float l[2], g[2];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            id[i] = j < k ? ids[j] : -1;
            if (id[i] < -1 || id[i] >= E) {
                bad = true;
                id[i] = -1;
            }
            l[i] = id[i] >= 0 ? as_logit(logits[id[i]]) : -INFINITY;
            g[i] = id[i] >= 0 && l[i] > -INFINITY ? a.scale * dw[j] : 0.f;
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0)
            atomicOr(a.err, MOE_DEVERR_BAD_EXPERT_ID);
        float term[2];           // what each chosen expert's entry gets
        float base = 0.f;        // softmax without renormalising: -sum_i dc_i p_i
        float mx = -INFINITY, inv_sum = 0.f;
        const bool dense = !a.sigmoid && !a.renormalize;
        if (a.renormalize) {
            // v = softmax of the chosen logits, or of their sigmoids' logarithms
            float z[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                z[i] = a.sigmoid ? fminf(l[i], 0.f) - log1pf(expf(-fabsf(l[i]))) : l[i];
            mx = warp_max(fmaxf(z[0], z[1]));
            float v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[i] = z[i] > -INFINITY ? expf(z[i] - mx) : 0.f;
            const float sum = warp_sum(v[0] + v[1]);
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
            v[0] *= inv;
            v[1] *= inv;
            const float dot = warp_sum(fmaf(g[0], v[0], g[1] * v[1]));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                term[i] = v[i] * (g[i] - dot);
                if (a.sigmoid)
                    term[i] *= 1.f / (1.f + expf(l[i]));
                if (v[i] == 0.f)
                    term[i] = 0.f;
            }
        } else if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float c = 1.f / (1.f + expf(-l[i]));
                term[i] = g[i] * c * (1.f / (1.f + expf(l[i])));
                if (g[i] == 0.f)
                    term[i] = 0.f;
            }
        } else {
            for (int e = lane; e < E; e += 32)
                mx = fmaxf(mx, as_logit(logits[e]));
            mx = warp_max(mx);
            float sum = 0.f;
            for (int e = lane; e < E; e += 32) {
                const float v = as_logit(logits[e]);
                sum += v > -INFINITY ? expf(v - mx) : 0.f;
            }
            sum = warp_sum(sum);
            inv_sum = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                term[i] = l[i] > -INFINITY ? g[i] * (expf(l[i] - mx) * inv_sum) : 0.f;
            base = -warp_sum(term[0] + term[1]);
        }
        // four consecutive experts a lane
        for (int e = 4 * lane; e < Ep; e += 128) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (dense)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E) {
                        const float x = as_logit(logits[e + i]);
                        v[i] = x > -INFINITY ? base * (expf(x - mx) * inv_sum) : 0.f;
                    }
            *reinterpret_cast<float4 *>(dl + e) = make_float4(v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
        for (int j = 0; j < k; ++j) {
            const int e = __shfl_sync(0xffffffffu, j < 32 ? id[0] : id[1], j & 31);
            const float v = __shfl_sync(0xffffffffu, j < 32 ? term[0] : term[1], j & 31);
            if (e >= 0 && ((e >> 2) & 31) == lane)
                dl[e] += v;
        }
        __syncwarp();
        __nv_bfloat16 *const parts = static_cast<__nv_bfloat16 *>(a.parts) + static_cast<size_t>(t) * 2 * Ep;
        const size_t at = static_cast<size_t>(t) * E;
        for (int e = 4 * lane; e < Ep; e += 128) {
            const float4 s4 = *reinterpret_cast<const float4 *>(dl + e);
            float v[4] = {s4.x, s4.y, s4.z, s4.w};
            if (whole && e < E) {         // E a multiple of 4: rows of whole 16-byte words
                if (a.d_logits_add) {
                    const float4 o = *reinterpret_cast<const float4 *>(a.d_logits_add + at + e);
                    v[0] += o.x;
                    v[1] += o.y;
                    v[2] += o.z;
                    v[3] += o.w;
                }
                if (a.d_logits)
                    *reinterpret_cast<float4 *>(a.d_logits + at + e) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E) {
                        if (a.d_logits_add)
                            v[i] += a.d_logits_add[at + e + i];
                        if (a.d_logits)
                            a.d_logits[at + e + i] = v[i];
                    }
            }
            __align__(8) __nv_bfloat16 hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[i] = __float2bfloat16_rn(v[i]);
                lo[i] = __float2bfloat16_rn(v[i] - __bfloat162float(hi[i]));
            }
            *reinterpret_cast<uint2 *>(parts + e) = *reinterpret_cast<const uint2 *>(hi);
            *reinterpret_cast<uint2 *>(parts + Ep + e) = *reinterpret_cast<const uint2 *>(lo);
        }
        __syncwarp();
    }
}

__global__ void __launch_bounds__(kThreads) sum_parts_kernel(const float4 *part, int parts, size_t n4,
                                                             void *out, int f32)
{
    pdl_wait();
    pdl_trigger();
    for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < n4;
         i += static_cast<size_t>(gridDim.x) * kThreads) {
        float4 sum = part[i];
        for (int p = 1; p < parts; ++p) {
            const float4 e = part[p * n4 + i];
            sum.x += e.x;
            sum.y += e.y;
            sum.z += e.z;
            sum.w += e.w;
        }
        if (f32) {
            static_cast<float4 *>(out)[i] = sum;
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
            uint2 o;
            o.x = *reinterpret_cast<const uint32_t *>(&lo);
            o.y = *reinterpret_cast<const uint32_t *>(&hi);
            static_cast<uint2 *>(out)[i] = o;
        }
    }
}

}  // namespace

cudaError_t launch_route_grad(const RouteGradArgs &a, int num_sms, cudaStream_t stream)
{
    const int Ep = (a.E + 63) & ~63;
    const long long need = (static_cast<long long>(a.T_max) + kThreads / 32 - 1) / (kThreads / 32);
    const long long most = num_sms * 8LL;
    return launch_k(route_grad_kernel, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(kThreads),
                    sizeof(float) * Ep * (kThreads / 32), stream, true, a);
}

cudaError_t launch_sum_parts(const float *part, int parts, size_t n, void *out, bool f32, int num_sms,
                             cudaStream_t stream)
{
    const size_t need = (n / 4 + kThreads - 1) / kThreads;
    const size_t most = num_sms * 8;
    return launch_k(sum_parts_kernel, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(kThreads), 0, stream,
                    true, reinterpret_cast<const float4 *>(part), parts, n / 4, out, f32 ? 1 : 0);
}

}  // namespace moe
