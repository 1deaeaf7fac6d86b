// norm_backward.cu -- gradient of the norm before the block, with the
// reduction of the weight's gradient.
//
//   x = h r w',  r = 1 / sqrt(mean(h^2) + eps),  w' = w or 1 + w
//   q = dx w',   dh = r (q - h r^2 mean(q h)) (+ dh_add),   dw = sum_t dx h r
//
// All sums in fp32. Bound by HBM: h, dx and dh_add are read once, dh is written
// once. As in the forward norm a row belongs to a group of threads that keeps
// it in registers; a thread meets the same columns in every row of its
// persistent block, so dw grows in registers, one fp32 sum a column, and each
// block ends with one row of partial sums. A second kernel adds those rows in
// order (deterministic: no atomics).
#include "moe_internal.h"
#include "norm_ops.cuh"

namespace moe {

namespace {

// Two sums over the tpr threads of a row group. s: one float2 per warp.
__device__ __forceinline__ float2 row_sums(Pair p, Pair q, int tpr, float2 *s)
{
    const float2 a = halves(p), b = halves(q);
    float u = a.x + a.y, v = b.x + b.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        u += __shfl_xor_sync(0xffffffffu, u, o);
        v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    if (tpr == 32)
        return make_float2(u, v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        s[warp] = make_float2(u, v);
    __syncthreads();
    const int n = tpr >> 5;      // at most 32
    const float2 w = lane < n ? s[warp / n * n + lane] : make_float2(0.f, 0.f);
    u = w.x;
    v = w.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        u += __shfl_xor_sync(0xffffffffu, u, o);
        v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return make_float2(u, v);
}

// Threads of a block and blocks of an SM: 16 columns a thread up to 1024
// threads, then 32 with the sums of dw in shared memory.
template <bool kF32, int kV, int kBlock>
struct GradPlan {
    static constexpr int kHeld = kV * Unit<kF32>::kCols;
    static constexpr bool kWide = kHeld > 16;
    static constexpr bool kAhead = !kWide && kBlock <= 512;
    static constexpr int kPerSm = kBlock == 256 ? 2 : 1;
};

template <bool kF32, int kV, int kBlock>
__global__ void __launch_bounds__(kBlock, GradPlan<kF32, kV, kBlock>::kPerSm)
    norm_backward_kernel(const __grid_constant__ NormGradArgs a, int tpr, float inv_H)
{
    using P = GradPlan<kF32, kV, kBlock>;
    using U = Unit<kF32>;
    constexpr int kCols = U::kCols, kPairs = U::kPairs;
    constexpr int kBytes = kF32 ? 4 : 2;
    extern __shared__ float4 s_dw4[];           // dw of the block's row groups (kWide: where it grows)
    __shared__ float2 s_sum[2][kBlock / 32];    // two, so that one barrier a row is enough
    float *const s_dw = reinterpret_cast<float *>(s_dw4);
    const int group = threadIdx.x / tpr, lane = threadIdx.x % tpr;
    const int rows = blockDim.x / tpr;
    int T = a.T_max;
    if (a.d_num_tokens) {
        T = *a.d_num_tokens;
        T = T < 0 ? 0 : (T > a.T_max ? a.T_max : T);
    }
    const int step = gridDim.x * rows;
    const int col0 = lane * kCols;
    bool on[kV];
    uint4 h[kV], more[kV];
    typename U::Half dx[kV];
    Pair acc[P::kWide ? 1 : kV][kPairs];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        on[v] = col0 + v * tpr * kCols < a.H;
        h[v] = more[v] = make_uint4(0u, 0u, 0u, 0u);
        dx[v] = typename U::Half{};
        if constexpr (!P::kWide) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                acc[v][i] = 0ull;
        } else if (on[v]) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                s_dw[col0 + v * tpr * kCols + i] = 0.f;
        }
    }
    auto load = [&](long long t) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (on[v]) {
                const int m = col0 + v * tpr * kCols;
                h[v] = ld_stream(static_cast<const char *>(a.h) + (t * a.h_stride + m) * kBytes);
                dx[v] = U::load_half(static_cast<const __nv_bfloat16 *>(a.dx) + t * a.dx_stride + m);
            }
    };
    int t = blockIdx.x * rows + group;
    if (P::kAhead && t < T)
        load(t);
    int turn = 0;
    for (int base = blockIdx.x * rows; base < T; base += step, t += step, turn ^= 1) {
        const bool row = t < T;
        if (!P::kAhead && row)
            load(t);
        if (a.dh_add && row) {
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (on[v])
                    more[v] = ld_stream(static_cast<const char *>(a.dh_add) +
                                        (t * a.add_stride + col0 + v * tpr * kCols) * kBytes);
        }
        Pair f[kV][kPairs], g[kV][kPairs];
        Pair hh = 0ull, qh = 0ull;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            U::pairs(h[v], f[v]);
            U::half_pairs(dx[v], g[v]);
        }
        if (P::kAhead && t + step < T)
            load(t + step);
        NormArgs wa;
        wa.w_f32 = a.w_f32;
        wa.unit_offset = a.unit_offset;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            Pair c[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                c[i] = g[v][i];
            if (on[v])
                U::times_weight(wa, a.w, col0 + v * tpr * kCols, c);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                hh = fma2(f[v][i], f[v][i], hh);
                qh = fma2(c[i], f[v][i], qh);
            }
        }
        const float2 sums = row_sums(hh, qh, tpr, s_sum[turn]);
        if (!row)
            continue;
        const float r = rsqrtf(fmaf(sums.x, inv_H, a.eps));
        const float k = -r * r * (sums.y * inv_H);
        const Pair r2 = pair(r, r), k2 = pair(k, k);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            if (!on[v])
                continue;
            const int m = col0 + v * tpr * kCols;
            Pair c[kPairs], o[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                c[i] = g[v][i];
            U::times_weight(wa, a.w, m, c);
            U::pairs(more[v], o);       // zero without dh_add
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                o[i] = fma2(r2, fma2(f[v][i], k2, c[i]), o[i]);
                const Pair n = mul2(f[v][i], r2);
                if constexpr (P::kWide) {
                    const float2 e = halves(mul2(g[v][i], n));
                    s_dw[m + 2 * i] += e.x;
                    s_dw[m + 2 * i + 1] += e.y;
                } else {
                    acc[v][i] = fma2(g[v][i], n, acc[v][i]);
                }
            }
            U::store(static_cast<char *>(a.dh) + (t * a.out_stride + m) * kBytes, o);
        }
    }
    if (!a.dw)
        return;
    // the block's row of partial sums: its groups' sums in group order
    if constexpr (!P::kWide) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (on[v])
#pragma unroll
                for (int i = 0; i < kPairs; ++i)
                    *reinterpret_cast<float2 *>(s_dw + group * a.H + col0 + v * tpr * kCols + 2 * i) = halves(acc[v][i]);
    }
    __syncthreads();
    for (int m = threadIdx.x * 4; m < a.H; m += blockDim.x * 4) {
        float4 sum = *reinterpret_cast<const float4 *>(s_dw + m);
        for (int gidx = 1; gidx < rows; ++gidx) {
            const float4 e = *reinterpret_cast<const float4 *>(s_dw + gidx * a.H + m);
            sum.x += e.x;
            sum.y += e.y;
            sum.z += e.z;
            sum.w += e.w;
        }
        *reinterpret_cast<float4 *>(a.part + static_cast<size_t>(blockIdx.x) * a.H + m) = sum;
    }
}

// dw[m] = sum of the partial rows: a block takes 32 x 4 columns, its warps
// every 32nd row each, then the warps' sums in order.
constexpr int kSumThreads = 1024;

__global__ void __launch_bounds__(kSumThreads) norm_dw_kernel(const float *__restrict__ part, int n, int H, void *dw,
                                                              int w_f32)
{
    __shared__ float4 s[kSumThreads / 32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = (blockIdx.x * 32 + lane) * 4;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m < H)
        for (int i = warp; i < n; i += kSumThreads / 32) {
            const float4 e = __ldg(reinterpret_cast<const float4 *>(part + static_cast<size_t>(i) * H + m));
            sum.x += e.x;
            sum.y += e.y;
            sum.z += e.z;
            sum.w += e.w;
        }
    s[warp][lane] = sum;
    __syncthreads();
    if (warp || m >= H)
        return;
    for (int i = 1; i < kSumThreads / 32; ++i) {
        const float4 e = s[i][lane];
        sum.x += e.x;
        sum.y += e.y;
        sum.z += e.z;
        sum.w += e.w;
    }
    if (w_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(dw) + m) = sum;
    else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
        uint2 o;
        o.x = *reinterpret_cast<const uint32_t *>(&lo);
        o.y = *reinterpret_cast<const uint32_t *>(&hi);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(dw) + m) = o;
    }
}

// Units of 16 bytes a thread holds, its row's threads and the block's.
struct GradShape {
    int v, tpr, block, per_sm;
    int rows() const { return block / tpr; }
    int grid(int T_max) const
    {
        const long long need = (static_cast<long long>(T_max) + rows() - 1) / rows();
        const long long most = 152LL * per_sm;    // a GB300's SMs; the workspace follows it
        return static_cast<int>(need < most ? need : most);
    }
};

GradShape grad_shape(int H, bool f32)
{
    const int units = H / (f32 ? 4 : 8);
    const int few = f32 ? 4 : 2;
    GradShape s;
    s.v = few;
    while (s.v > 1 && units / s.v < 32)
        s.v /= 2;
    if (units > 1024 * s.v)
        s.v = 2 * few;
    s.tpr = ((units + s.v - 1) / s.v + 31) / 32 * 32;
    s.block = s.tpr <= 256 ? 256 / s.tpr * s.tpr : s.tpr;
    s.per_sm = s.tpr <= 256 ? 2 : 1;
    return s;
}

template <bool kF32, int kV, int kBlock>
cudaError_t run(const NormGradArgs &a, const GradShape &s, cudaStream_t stream)
{
    auto kern = norm_backward_kernel<kF32, kV, kBlock>;
    const size_t smem = a.dw || GradPlan<kF32, kV, kBlock>::kWide ? sizeof(float) * s.rows() * a.H : 0;
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
        if (e != cudaSuccess)
            return e;
    }
    return launch_k(kern, dim3(s.grid(a.T_max)), dim3(s.block), smem, stream, false, a, s.tpr, 1.f / a.H);
}

template <bool kF32>
cudaError_t run_units(const NormGradArgs &a, const GradShape &s, cudaStream_t stream)
{
    constexpr int kFew = kF32 ? 4 : 2;
    if (s.v == 2 * kFew)
        return run<kF32, 2 * kFew, 1024>(a, s, stream);
    if (s.v == kFew)
        return s.tpr <= 256 ? run<kF32, kFew, 256>(a, s, stream)
                            : (s.tpr <= 512 ? run<kF32, kFew, 512>(a, s, stream)
                                            : run<kF32, kFew, 1024>(a, s, stream));
    if (kF32 && s.v == 2)
        return run<kF32, 2, 256>(a, s, stream);
    return run<kF32, 1, 256>(a, s, stream);
}

}  // namespace

int norm_grad_part_rows(int T_max, int H, bool h_f32) { return grad_shape(H, h_f32).grid(T_max); }

cudaError_t launch_norm_backward(const NormGradArgs &a, cudaStream_t stream)
{
    const GradShape s = grad_shape(a.H, a.h_f32);
    const cudaError_t e = a.h_f32 ? run_units<true>(a, s, stream) : run_units<false>(a, s, stream);
    if (e != cudaSuccess || !a.dw)
        return e;
    return launch_k(norm_dw_kernel, dim3((a.H + 127) / 128), dim3(kSumThreads), 0, stream, false,
                    static_cast<const float *>(a.part), s.grid(a.T_max), a.H, a.dw, a.w_f32);
}

}  // namespace moe
