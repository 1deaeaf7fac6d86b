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
// show in an fp32 dw_router only. T=8192, E=128, H=4096 46 us in a graph (0.15 GB, 22 us
// at the copy rate): 6 us for dl, then the two products, 19 and 17 us on their own,
// which end in epilogues of a few K blocks' work each, then 4 for the sum of
// dw_router's four token ranges. A few slots go another way (route_grad_few_kernel).
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

// The chosen experts of token t and their terms of dl, by a warp: slots lane and
// lane + 32 (id -1: none). Softmax without renormalising also has a term for
// every expert: p_e times `base`, p_e = exp(l_e - mx) inv_sum.
struct Chosen {
    int id[2];
    float term[2];
    float base, mx, inv_sum;
};

__device__ __forceinline__ Chosen chosen_terms(const RouteGradArgs &a, int t)
{
    const int lane = threadIdx.x & 31, E = a.E, k = a.k;
    const float *const logits = a.logits + static_cast<size_t>(t) * E;
    const int32_t *const ids = a.ids + static_cast<size_t>(t) * k;
    const float *const dw = a.d_weights + static_cast<size_t>(t) * k;
    Chosen c;
    float l[2], g[2];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        c.id[i] = j < k ? ids[j] : -1;
        const float d = j < k ? dw[j] : 0.f;
        if (c.id[i] < -1 || c.id[i] >= E) {
            bad = true;
            c.id[i] = -1;
        }
        l[i] = c.id[i] >= 0 ? as_logit(logits[c.id[i]]) : -INFINITY;
        g[i] = l[i] > -INFINITY ? a.scale * d : 0.f;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0)
        atomicOr(a.err, MOE_DEVERR_BAD_EXPERT_ID);
    c.base = 0.f;
    c.mx = -INFINITY;
    c.inv_sum = 0.f;
    if (a.renormalize) {
        // v = softmax of the chosen logits, or of their sigmoids' logarithms
        float z[2], v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            z[i] = a.sigmoid ? fminf(l[i], 0.f) - log1pf(expf(-fabsf(l[i]))) : l[i];
        const float mx = warp_max(fmaxf(z[0], z[1]));
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
            c.term[i] = v[i] * (g[i] - dot);
            if (a.sigmoid)
                c.term[i] *= 1.f / (1.f + expf(l[i]));
            if (v[i] == 0.f)
                c.term[i] = 0.f;
        }
    } else if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float p = 1.f / (1.f + expf(-l[i]));
            c.term[i] = g[i] == 0.f ? 0.f : g[i] * p * (1.f / (1.f + expf(l[i])));
        }
    } else {
        for (int e = lane; e < E; e += 32)
            c.mx = fmaxf(c.mx, as_logit(logits[e]));
        c.mx = warp_max(c.mx);
        float sum = 0.f;
        for (int e = lane; e < E; e += 32) {
            const float v = as_logit(logits[e]);
            sum += v > -INFINITY ? expf(v - c.mx) : 0.f;
        }
        sum = warp_sum(sum);
        c.inv_sum = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c.term[i] = l[i] > -INFINITY ? g[i] * (expf(l[i] - c.mx) * c.inv_sum) : 0.f;
        c.base = -warp_sum(c.term[0] + c.term[1]);
    }
    return c;
}

__device__ __forceinline__ int token_count(const RouteGradArgs &a)
{
    if (!a.d_num_tokens)
        return a.T_max;
    const int T = *a.d_num_tokens;
    return T < 0 ? 0 : (T > a.T_max ? a.T_max : T);
}

// Adds the chosen experts' terms to a token's row dl[] in shared memory, slot by
// slot, each by the lane that owns the expert's word (experts in fours).
__device__ __forceinline__ void add_terms(float *dl, const Chosen &c, int k)
{
    for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(0xffffffffu, j < 32 ? c.id[0] : c.id[1], j & 31);
        const float v = __shfl_sync(0xffffffffu, j < 32 ? c.term[0] : c.term[1], j & 31);
        if (e >= 0 && ((e >> 2) & 31) == static_cast<int>(threadIdx.x & 31))
            dl[e] += v;
    }
}

// The leading bf16 part of an element of dl. One that would round up to infinity is
// cut off instead, its rest then holds what is missing; an infinite one has no rest.
__device__ __forceinline__ __nv_bfloat16 leading_part(float v)
{
    return fabsf(v) > 3.38953139e38f ? __float2bfloat16_rz(v) : __float2bfloat16_rn(v);     // the largest bf16
}

// One warp per token. Its row of dl grows in shared memory: base values, then
// the chosen experts' terms.
__global__ void __launch_bounds__(kThreads) route_grad_kernel(const __grid_constant__ RouteGradArgs a)
{
    extern __shared__ float4 s_row[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, k = a.k, Ep = (E + 63) & ~63;
    const bool whole = E % 4 == 0;
    float *const dl = reinterpret_cast<float *>(s_row) + warp * Ep;
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < Ep; i += kThreads)     // 2 Ep bf16 zeros
            reinterpret_cast<uint32_t *>(a.parts)[static_cast<size_t>(a.T_max) * Ep + i] = 0u;
    for (int t = blockIdx.x * (kThreads / 32) + warp; t < T; t += gridDim.x * (kThreads / 32)) {
        const float *const logits = a.logits + static_cast<size_t>(t) * E;
        const Chosen c = chosen_terms(a, t);
        const bool dense = !a.sigmoid && !a.renormalize;
        // four consecutive experts a lane
        for (int e = 4 * lane; e < Ep; e += 128) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (dense)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E) {
                        const float x = as_logit(logits[e + i]);
                        v[i] = x > -INFINITY ? c.base * (expf(x - c.mx) * c.inv_sum) : 0.f;
                    }
            *reinterpret_cast<float4 *>(dl + e) = make_float4(v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
        add_terms(dl, c, k);
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
                hi[i] = leading_part(v[i]);
                lo[i] = isinf(v[i]) ? __float2bfloat16_rn(0.f) : __float2bfloat16_rn(v[i] - __bfloat162float(hi[i]));
            }
            *reinterpret_cast<uint2 *>(parts + e) = *reinterpret_cast<const uint2 *>(hi);
            *reinterpret_cast<uint2 *>(parts + Ep + e) = *reinterpret_cast<const uint2 *>(lo);
        }
        __syncwarp();
    }
}

// A few slots whose dl is zero but at the chosen experts (sigmoid or
// renormalised scores, no gradient added): dx and dw_router are sums of T * k
// rows in fp32, in one kernel, where the products on the tensor cores take two
// kernels of some 3 and 11 us whatever their size. Blocks of 1024 columns:
//  * of a token's dx: its k terms, then k rows of w_router;
//  * of an expert's dw_router: the slots that chose it, found in order among all
//    of them, their terms, then their rows of x; an expert without slots gets zeros;
//  * d_logits: four tokens a block.
constexpr int kFewThreads = 128;

__device__ __forceinline__ void fma8(float (&acc)[8], float c, const uint4 &u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(c, __uint_as_float(w[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(c, __uint_as_float(w[i] & 0xffff0000u), acc[2 * i + 1]);
    }
}

__device__ __forceinline__ void store8(void *out, size_t at, bool f32, const float (&v)[8])
{
    if (f32) {
        float4 *const p = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The term of one slot (sigmoid or renormalised scores), by one thread: many
// slots of an expert are worked out side by side.
__device__ __forceinline__ float slot_term(const RouteGradArgs &a, int slot)
{
    const int k = a.k, t = slot / k;
    const float *const logits = a.logits + static_cast<size_t>(t) * a.E;
    const int32_t *const ids = a.ids + static_cast<size_t>(t) * k;
    const float *const dw = a.d_weights + static_cast<size_t>(t) * k;
    const float l = as_logit(logits[ids[slot - t * k]]), g = a.scale * dw[slot - t * k];
    if (!(l > -INFINITY))
        return 0.f;
    if (!a.renormalize)
        return g * (1.f / (1.f + expf(-l))) * (1.f / (1.f + expf(l)));
    auto z_of = [&](int j) {
        const int e = ids[j];
        const float v = e >= 0 && e < a.E ? as_logit(logits[e]) : -INFINITY;
        return a.sigmoid ? fminf(v, 0.f) - log1pf(expf(-fabsf(v))) : v;
    };
    float mx = -INFINITY;
    for (int j = 0; j < k; ++j)
        mx = fmaxf(mx, z_of(j));
    float sum = 0.f, dot = 0.f;
    for (int j = 0; j < k; ++j) {
        const float z = z_of(j), v = z > -INFINITY ? expf(z - mx) : 0.f;
        sum += v;
        if (v > 0.f)
            dot = fmaf(a.scale * dw[j], v, dot);
    }
    const float v = expf((a.sigmoid ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l) - mx) / sum;
    const float term = v * (g - dot / sum);
    return v == 0.f ? 0.f : (a.sigmoid ? term * (1.f / (1.f + expf(l))) : term);
}

__global__ void __launch_bounds__(kFewThreads) route_grad_few_kernel(const __grid_constant__ RouteGradArgs a,
                                                                     const __grid_constant__ RouteFewArgs f)
{
    __shared__ int s_id[kRouteFewSlots];
    __shared__ float s_term[kRouteFewSlots];
    __shared__ int s_count[kFewThreads / 32];
    extern __shared__ float4 s_few[];             // d_logits: four rows of E floats, rounded up to fours
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, k = a.k, H = f.H, chunks = (H + 1023) / 1024;
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a);
    int b = blockIdx.x;
    const int dx_blocks = f.dx ? a.T_max * chunks : 0, dw_blocks = f.dw ? E * chunks : 0;
    if (b < dx_blocks) {
        const int t = b / chunks, m = (b % chunks) * 1024 + 8 * threadIdx.x;
        if (t >= T)
            return;
        if (warp == 0) {
            const Chosen c = chosen_terms(a, t);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (lane + 32 * i < k) {
                    s_id[lane + 32 * i] = c.id[i];
                    s_term[lane + 32 * i] = c.term[i];
                }
        }
        __syncthreads();
        if (m >= H)
            return;
        float acc[8] = {};
#pragma unroll 4
        for (int j = 0; j < k; ++j)
            if (s_id[j] >= 0)
                fma8(acc, s_term[j],
                     __ldg(reinterpret_cast<const uint4 *>(f.w + static_cast<size_t>(s_id[j]) * H + m)));
        store8(f.dx, static_cast<size_t>(t) * H + m, false, acc);
        return;
    }
    b -= dx_blocks;
    if (b < dw_blocks) {
        const int e = b / chunks, m = (b % chunks) * 1024 + 8 * threadIdx.x;
        // the slots of this expert, ascending
        const int slots = T * k;
        int found = 0;
        for (int s0 = 0; s0 < slots; s0 += kFewThreads) {
            const int s = s0 + static_cast<int>(threadIdx.x);
            const int id = s < slots ? a.ids[s] : -1;
            if (e == 0 && (id < -1 || id >= E))
                atomicOr(a.err, MOE_DEVERR_BAD_EXPERT_ID);     // slot_term does not report it
            const bool hit = id == e;
            const unsigned hits = __ballot_sync(0xffffffffu, hit);
            if (lane == 0)
                s_count[warp] = __popc(hits);
            __syncthreads();
            int at = found;
#pragma unroll
            for (int w = 0; w < kFewThreads / 32; ++w) {
                if (w < warp)
                    at += s_count[w];
                found += s_count[w];
            }
            if (hit)
                s_id[at + __popc(hits & ((1u << lane) - 1))] = s;
            __syncthreads();
        }
        if (found <= kFewThreads / 32) {
            if (warp < found) {            // a warp each: 1.2 us, slot_term 2 us
                const int s = s_id[warp], t = s / k, j = s - t * k;
                const Chosen c = chosen_terms(a, t);
                const float v = __shfl_sync(0xffffffffu, j < 32 ? c.term[0] : c.term[1], j & 31);
                if (lane == 0) {
                    s_term[warp] = v;
                    s_id[warp] = t;        // from here on the slot's token
                }
            }
        } else {
            for (int i = threadIdx.x; i < found; i += kFewThreads) {
                s_term[i] = slot_term(a, s_id[i]);
                s_id[i] /= k;
            }
        }
        __syncthreads();
        if (m >= H)
            return;
        float acc[8] = {};
        for (int i0 = 0; i0 < found; i0 += 8) {
            uint4 row[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < found)
                    row[i] = __ldg(reinterpret_cast<const uint4 *>(f.x + static_cast<size_t>(s_id[i0 + i]) * H + m));
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < found)
                    fma8(acc, s_term[i0 + i], row[i]);
        }
        store8(f.dw, static_cast<size_t>(e) * H + m, f.dw_f32 != 0, acc);
        return;
    }
    b -= dw_blocks;
    // d_logits of four tokens
    const int E4 = (E + 3) & ~3;
    float *const dl = reinterpret_cast<float *>(s_few) + warp * E4;
    const int t = b * (kFewThreads / 32) + warp;
    if (t >= T)
        return;
    const Chosen c = chosen_terms(a, t);
    for (int e = 4 * lane; e < E4; e += 128)
        *reinterpret_cast<float4 *>(dl + e) = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
    add_terms(dl, c, k);
    __syncwarp();
    for (int e = lane; e < E; e += 32)
        a.d_logits[static_cast<size_t>(t) * E + e] = dl[e];
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

cudaError_t launch_route_grad_few(const RouteGradArgs &a, const RouteFewArgs &f, cudaStream_t stream)
{
    const int chunks = (f.H + 1023) / 1024, warps = kFewThreads / 32;
    const long long blocks = (f.dx ? static_cast<long long>(a.T_max) * chunks : 0) +
                             (f.dw ? static_cast<long long>(a.E) * chunks : 0) +
                             (a.d_logits ? (a.T_max + warps - 1) / warps : 0);
    return launch_k(route_grad_few_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads),
                    a.d_logits ? sizeof(float) * ((a.E + 3) & ~3) * warps : 0, stream, true, a, f);
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
