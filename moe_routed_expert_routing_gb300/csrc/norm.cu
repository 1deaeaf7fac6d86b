// norm.cu -- the norm of the residual stream before the block, and the way
// back into it after the block: norm of the block's output, gate, residual
// scale, and the next block's norm in the same pass.
//
//   moe_norm:           x = h * r(h) * w
//   moe_norm_residual:  h' = h + s * g * (y * r(y) * w_post),  x_next = h' * r(h') * w_next
//   r(v) = 1 / sqrt(mean(v^2) + eps)
//
// All sums and products in fp32, one rounding per output. Bound by HBM: every
// input is read once and every output written once. A row belongs to a group
// of 32..512 threads that keeps it in registers from the load to the store,
// so the row sums cost no second read. Blocks are persistent and load their
// next row before the sums of this one, so loads are in flight through the
// barriers; the weights stay in L1 (the streams are loaded past it).
#include <type_traits>

#include <cuda_bf16.h>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kMaxBlock = 512;

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

__device__ __forceinline__ void widen(uint32_t u, float &lo, float &hi)
{
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xffff0000u);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// A thread's unit is 16 bytes of the residual stream: 8 columns of bf16 or 4 of fp32.
template <bool kF32>
struct Unit {
    static constexpr int kCols = kF32 ? 4 : 8;
    using Half = typename std::conditional<kF32, uint2, uint4>::type;   // the same columns in bf16

    static __device__ __forceinline__ Half load_half(const __nv_bfloat16 *p)
    {
        if constexpr (kF32)
            return ld_stream2(p);
        else
            return ld_stream(p);
    }

    static __device__ __forceinline__ void floats(const uint4 &u, float (&f)[kCols])
    {
        if constexpr (kF32) {
            f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
            f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
        } else {
            widen(u.x, f[0], f[1]); widen(u.y, f[2], f[3]);
            widen(u.z, f[4], f[5]); widen(u.w, f[6], f[7]);
        }
    }

    static __device__ __forceinline__ void half_floats(const Half &u, float (&f)[kCols])
    {
        widen(u.x, f[0], f[1]);
        widen(u.y, f[2], f[3]);
        if constexpr (!kF32) {
            widen(u.z, f[4], f[5]);
            widen(u.w, f[6], f[7]);
        }
    }

    static __device__ __forceinline__ void store_half(__nv_bfloat16 *p, const float (&f)[kCols])
    {
        if constexpr (kF32)
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack(f[0], f[1]), pack(f[2], f[3]));
        else
            *reinterpret_cast<uint4 *>(p) =
                make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
    }

    static __device__ __forceinline__ void store(void *p, const float (&f)[kCols])
    {
        if constexpr (kF32)
            *static_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        else
            store_half(static_cast<__nv_bfloat16 *>(p), f);
    }

    // kCols values of a per-channel vector of either type
    static __device__ __forceinline__ void channel(const void *p, bool f32, int m, float (&f)[kCols])
    {
        if (f32) {
#pragma unroll
            for (int i = 0; i < kCols; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + m + i));
                f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
            }
        } else {
            half_floats(__ldg(reinterpret_cast<const Half *>(static_cast<const __nv_bfloat16 *>(p) + m)), f);
        }
    }
};

template <bool kF32>
__device__ __forceinline__ void norm_weight(const NormArgs &a, const void *w, int m, float (&f)[Unit<kF32>::kCols])
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < Unit<kF32>::kCols; ++i)
            f[i] = 1.f;
        return;
    }
    Unit<kF32>::channel(w, a.w_f32, m, f);
    if (a.unit_offset)
#pragma unroll
        for (int i = 0; i < Unit<kF32>::kCols; ++i)
            f[i] += 1.f;
}

// Sum over the tpr threads of a row group (whole warps); every thread of the
// block calls it. s: this sum's words, one per warp of the block.
__device__ __forceinline__ float row_sum(float v, int tpr, float *s)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32)
        return v;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
        s[warp] = v;
    __syncthreads();
    const int n = tpr >> 5, first = warp / n * n;
    v = 0.f;
    for (int i = 0; i < n; ++i)
        v += s[first + i];
    return v;
}

// Whether an instance fits 64 registers with its next row in them: two blocks
// of 512 threads on an SM then. The wider rows run one block and load late.
template <bool kF32, int kV, bool kRes>
constexpr bool kLean = kV <= 2 || (kV == 4 && (kF32 || !kRes));

// kV units per thread; kRes: moe_norm_residual. tpr threads per row.
template <bool kF32, int kV, bool kRes>
__global__ void __launch_bounds__(kMaxBlock, kLean<kF32, kV, kRes> ? 2 : 1) norm_kernel(const __grid_constant__ NormArgs a, int tpr)
{
    using U = Unit<kF32>;
    constexpr int kCols = U::kCols;
    constexpr bool kAhead = kLean<kF32, kV, kRes>;   // the next row in registers too
    // two buffers: a row's words are not written again before every thread
    // has passed the barrier of the other sum
    __shared__ float s_sum[2][kMaxBlock / 32];
    const int group = threadIdx.x / tpr, lane = threadIdx.x % tpr;
    const int rows = blockDim.x / tpr;
    const int units = a.H / kCols;
    pdl_wait();
    pdl_trigger();
    int T = a.T_max;
    if (a.d_num_tokens) {
        T = *a.d_num_tokens;
        T = T < 0 ? 0 : (T > a.T_max ? a.T_max : T);
    }
    uint4 h[kV];
    typename U::Half y[kRes ? kV : 1];
    auto load = [&](long long t) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int u = lane + v * tpr;
            if (t < T && u < units) {
                h[v] = ld_stream(static_cast<const char *>(a.h) + (t * a.h_stride + u * kCols) * (kF32 ? 4 : 2));
                if constexpr (kRes)
                    y[v] = U::load_half(static_cast<const __nv_bfloat16 *>(a.y) + t * a.y_stride + u * kCols);
            }
        }
    };
    const long long step = static_cast<long long>(gridDim.x) * rows;
    long long base = static_cast<long long>(blockIdx.x) * rows;
    if (kAhead)
        load(base + group);
    for (; base < T; base += step) {
        const long long t = base + group;
        if (!kAhead)
            load(t);
        const bool row = t < T;
        float f[kV][kCols];
        if constexpr (kRes) {
            float n[kV][kCols];
            float q = 0.f;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                U::floats(h[v], f[v]);
                U::half_floats(y[v], n[v]);
                if (row && lane + v * tpr < units)
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        q = fmaf(n[v][i], n[v][i], q);
            }
            if (kAhead)
                load(t + step);
            const float r = a.norm_block ? 1.f / sqrtf(row_sum(q, tpr, s_sum[0]) / a.H + a.eps) : 1.f;
            const float s = (row && a.gate_kind == MOE_GATE_TOKEN ? static_cast<const float *>(a.gate)[t] : 1.f) * a.scale;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int u = lane + v * tpr;
                if (!row || u >= units)
                    continue;
                float c[kCols];
                if (a.norm_block) {
                    norm_weight<kF32>(a, a.w_post, u * kCols, c);
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        n[v][i] *= r * c[i];
                }
                if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT) {
                    if (a.gate_kind == MOE_GATE_CHANNEL)
                        U::channel(a.gate, a.w_f32, u * kCols, c);
                    else
                        U::half_floats(U::load_half(static_cast<const __nv_bfloat16 *>(a.gate) + t * a.gate_stride +
                                                    u * kCols), c);
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        n[v][i] *= c[i];
                }
#pragma unroll
                for (int i = 0; i < kCols; ++i)
                    f[v][i] = fmaf(s, n[v][i], f[v][i]);
                U::store(static_cast<char *>(a.h_out) + (t * a.out_stride + u * kCols) * (kF32 ? 4 : 2), f[v]);
            }
            if (!a.x) {
                if (tpr != 32)
                    __syncthreads();   // s_sum[0] is free for the next row
                continue;
            }
        } else {
#pragma unroll
            for (int v = 0; v < kV; ++v)
                U::floats(h[v], f[v]);
            if (kAhead)
                load(t + step);
        }
        float q = 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (row && lane + v * tpr < units)
#pragma unroll
                for (int i = 0; i < kCols; ++i)
                    q = fmaf(f[v][i], f[v][i], q);
        const float r = 1.f / sqrtf(row_sum(q, tpr, s_sum[1]) / a.H + a.eps);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int u = lane + v * tpr;
            if (!row || u >= units)
                continue;
            float c[kCols];
            norm_weight<kF32>(a, a.w_next, u * kCols, c);
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                f[v][i] *= r * c[i];
            U::store_half(static_cast<__nv_bfloat16 *>(a.x) + t * a.x_stride + u * kCols, f[v]);
        }
        if ((!kRes || !a.norm_block) && tpr != 32)
            __syncthreads();   // one sum per row: s_sum[1] is free for the next row
    }
}

template <bool kF32, int kV>
cudaError_t launch(const NormArgs &a, int tpr, int num_sms, cudaStream_t stream, bool pdl)
{
    const int rows = tpr < 256 ? 256 / tpr : 1;
    const int threads = rows * tpr;
    const long long need = (static_cast<long long>(a.T_max) + rows - 1) / rows;
    const long long most = static_cast<long long>(num_sms) * (1024 / threads);
    const dim3 grid(static_cast<unsigned>(need < most ? need : most));
    return a.y ? launch_k(norm_kernel<kF32, kV, true>, grid, dim3(threads), 0, stream, pdl, a, tpr)
               : launch_k(norm_kernel<kF32, kV, false>, grid, dim3(threads), 0, stream, pdl, a, tpr);
}

template <bool kF32>
cudaError_t launch_units(const NormArgs &a, int num_sms, cudaStream_t stream, bool pdl)
{
    // 32 bytes (bf16) or 64 bytes (fp32) of the stream per thread, fewer where
    // a row would not fill a warp, more where it would need over 512 threads
    const int units = a.H / Unit<kF32>::kCols;
    int v = kF32 ? 4 : 2;
    while (v > 1 && units / v < 32)
        v /= 2;
    while ((units + v - 1) / v > kMaxBlock)
        v *= 2;
    const int tpr = ((units + v - 1) / v + 31) / 32 * 32;
    switch (v) {
    case 1:
        return launch<kF32, 1>(a, tpr, num_sms, stream, pdl);
    case 2:
        return launch<kF32, 2>(a, tpr, num_sms, stream, pdl);
    case 4:
        return launch<kF32, 4>(a, tpr, num_sms, stream, pdl);
    case 8:
        return launch<kF32, 8>(a, tpr, num_sms, stream, pdl);
    default:
        return launch<kF32, 16>(a, tpr, num_sms, stream, pdl);
    }
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t stream, bool pdl)
{
    return a.h_f32 ? launch_units<true>(a, num_sms, stream, pdl) : launch_units<false>(a, num_sms, stream, pdl);
}

}  // namespace moe
