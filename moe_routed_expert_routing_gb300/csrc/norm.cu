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
// barriers; the weights stay in L1 (the streams are loaded past it). The
// arithmetic runs on packed pairs (fma.rn.f32x2): at HBM's pace an SM has
// about 12 issue slots for 32 elements of bf16, and scalar arithmetic with a
// division and a square root per thread and row took 74% of all issue slots
// (T=8192, H=4096, bf16: 25.0 us on one buffer, part of which stays in L2; with
// the residual in fp32 87 us). Now 43%: 22.5 us so, 25.1 us on inputs larger than
// L2 (0.79 of the measured copy rate; fp32 33.3, 0.89); 68.5 us, 0.87 (T=8191, fp32
// stream, channel gate, next norm). One row of 7168: 2.5 us, the launch. Longer rows hold
// 32 columns a thread and take their factors from L1: T=8192, H=7168 50.1 us (0.69
// of the copy rate; fp32 60.1, 0.87), with the residual 108 (0.64; fp32 162, 0.64).
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

// Blocks of kBlock threads that share an SM, by the columns a thread holds.
// Per-channel factors stay in registers where they leave two blocks or more an
// SM: 16 columns with the residual, T=8191 of 4096 in fp32, 68.5 us so in two
// blocks and 72.8 with the factors from L1 in three.
template <bool kF32, int kV, bool kRes, int kBlock>
struct Plan {
    static constexpr int kHeld = kV * Unit<kF32>::kCols;
    static constexpr bool kAhead = kHeld <= 32;   // the next row in registers too
    static constexpr bool kKeep = kHeld <= 16;    // and the per-channel factors
    static constexpr int kPerSm =
        kBlock == 256 ? (kHeld <= 8 ? (kRes ? 3 : 4) : (kHeld <= 16 ? (kRes ? 2 : 3) : 2)) : (kHeld <= 16 && !kRes ? 2 : 1);
};

// kV units per thread; kRes: moe_norm_residual. tpr threads per row.
template <bool kF32, int kV, bool kRes, int kBlock>
__global__ void __launch_bounds__(kBlock, Plan<kF32, kV, kRes, kBlock>::kPerSm)
    norm_kernel(const __grid_constant__ NormArgs a, int tpr, float inv_H)
{
    using U = Unit<kF32>;
    constexpr int kCols = U::kCols, kPairs = U::kPairs;
    constexpr int kBytes = kF32 ? 4 : 2;
    constexpr bool kAhead = Plan<kF32, kV, kRes, kBlock>::kAhead;
    // two buffers: a row's words are not written again before every thread
    // has passed the barrier of the other sum
    __shared__ float s_sum[2][kBlock / 32];
    const int group = threadIdx.x / tpr, lane = threadIdx.x % tpr;
    const int rows = blockDim.x / tpr;
    pdl_wait();
    pdl_trigger();
    int T = a.T_max;
    if (a.d_num_tokens) {
        T = *a.d_num_tokens;
        T = T < 0 ? 0 : (T > a.T_max ? a.T_max : T);
    }
    const int step = gridDim.x * rows;
    int t = blockIdx.x * rows + group;
    // this thread's first column of its next row in each tensor
    const int col0 = lane * kCols;
    const char *h_at = static_cast<const char *>(a.h) + (t * a.h_stride + col0) * kBytes;
    const __nv_bfloat16 *y_at = static_cast<const __nv_bfloat16 *>(a.y) + t * a.y_stride + col0;
    bool on[kV];      // columns past H: never loaded, zero
    uint4 h[kV];
    typename U::Half y[kRes ? kV : 1];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        on[v] = col0 + v * tpr * kCols < a.H;
        h[v] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (kRes)
            y[v] = typename U::Half{};
    }
    // per-channel factors: of y, s * w_post' * channel gate; of the normed row, w_next'
    auto factors_y = [&](int v, Pair(&c)[kPairs]) {
        const int m = col0 + v * tpr * kCols;
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            c[i] = pair(a.scale, a.scale);
        if (a.norm_block)
            U::times_weight(a, a.w_post, m, c);
        if (a.gate_kind == MOE_GATE_CHANNEL) {
            Pair g[kPairs];
            U::channel(a.gate, a.w_f32, m, g);
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                c[i] = mul2(c[i], g[i]);
        }
    };
    auto factors_x = [&](int v, Pair(&c)[kPairs]) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            c[i] = pair(1.f, 1.f);
        U::times_weight(a, a.w_next, col0 + v * tpr * kCols, c);
    };
    constexpr bool kKeep = Plan<kF32, kV, kRes, kBlock>::kKeep;
    Pair keep_y[kKeep && kRes ? kV : 1][kPairs], keep_x[kKeep ? kV : 1][kPairs];
    if constexpr (kKeep) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (on[v]) {
                if constexpr (kRes)
                    factors_y(v, keep_y[v]);
                if (a.x)
                    factors_x(v, keep_x[v]);
            }
    }
    auto load = [&]() {
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (on[v]) {
                h[v] = ld_stream(h_at + v * tpr * kCols * kBytes);
                if constexpr (kRes)
                    y[v] = U::load_half(y_at + v * tpr * kCols);
            }
        h_at += step * a.h_stride * kBytes;
        if constexpr (kRes)
            y_at += step * a.y_stride;
    };
    if (kAhead && t < T)
        load();
    for (int base = blockIdx.x * rows; base < T; base += step, t += step) {
        const bool row = t < T;
        if (!kAhead && row)
            load();
        Pair f[kV][kPairs];
        if constexpr (kRes) {
            Pair n[kV][kPairs];
            Pair q = 0ull;
            float r = 1.f;       // what a row's y is multiplied by
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                U::pairs(h[v], f[v]);
                U::half_pairs(y[v], n[v]);
            }
            if (kAhead && t + step < T)
                load();
            if (a.norm_block) {
#pragma unroll
                for (int v = 0; v < kV; ++v)
#pragma unroll
                    for (int i = 0; i < kPairs; ++i)
                        q = fma2(n[v][i], n[v][i], q);
                r = rsqrtf(fmaf(row_sum(q, tpr, s_sum[0]), inv_H, a.eps));
            }
            if (row) {
                if (a.gate_kind == MOE_GATE_TOKEN)
                    r *= static_cast<const float *>(a.gate)[t];
                const Pair r2 = pair(r, r);
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    const int m = col0 + v * tpr * kCols;
                    if (!on[v])
                        continue;
                    Pair c[kPairs];
                    if constexpr (kKeep) {
#pragma unroll
                        for (int i = 0; i < kPairs; ++i)
                            c[i] = keep_y[v][i];
                    } else {
                        factors_y(v, c);
                    }
                    if (a.gate_kind == MOE_GATE_ELEMENT) {
                        Pair g[kPairs];
                        U::half_pairs(U::load_half(static_cast<const __nv_bfloat16 *>(a.gate) + t * a.gate_stride + m), g);
#pragma unroll
                        for (int i = 0; i < kPairs; ++i)
                            c[i] = mul2(c[i], g[i]);
                    }
#pragma unroll
                    for (int i = 0; i < kPairs; ++i)
                        f[v][i] = fma2(mul2(n[v][i], r2), c[i], f[v][i]);
                    U::store(static_cast<char *>(a.h_out) + (t * a.out_stride + m) * kBytes, f[v]);
                }
            }
            if (!a.x) {
                if (tpr != 32)
                    __syncthreads();   // s_sum[0] is free for the next row
                continue;
            }
        } else {
#pragma unroll
            for (int v = 0; v < kV; ++v)
                U::pairs(h[v], f[v]);
            if (kAhead && t + step < T)
                load();
        }
        Pair q = 0ull;
#pragma unroll
        for (int v = 0; v < kV; ++v)
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                q = fma2(f[v][i], f[v][i], q);
        const float r = rsqrtf(fmaf(row_sum(q, tpr, s_sum[1]), inv_H, a.eps));
        if (row) {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int m = col0 + v * tpr * kCols;
                if (!on[v])
                    continue;
                Pair c[kPairs];
                if constexpr (kKeep) {
#pragma unroll
                    for (int i = 0; i < kPairs; ++i)
                        c[i] = keep_x[v][i];
                } else {
                    factors_x(v, c);
                }
                const Pair r2 = pair(r, r);
#pragma unroll
                for (int i = 0; i < kPairs; ++i)
                    f[v][i] = mul2(mul2(f[v][i], r2), c[i]);
                U::store_half(static_cast<__nv_bfloat16 *>(a.x) + t * a.x_stride + m, f[v]);
            }
        }
        if ((!kRes || !a.norm_block) && tpr != 32)
            __syncthreads();   // one sum per row: s_sum[1] is free for the next row
    }
}

template <bool kF32, int kV, bool kRes, int kBlock>
cudaError_t launch(const NormArgs &a, int tpr, int num_sms, cudaStream_t stream, bool pdl)
{
    const int rows = kBlock == 256 ? 256 / tpr : 1;
    const long long need = (static_cast<long long>(a.T_max) + rows - 1) / rows;
    const long long most = static_cast<long long>(num_sms) * Plan<kF32, kV, kRes, kBlock>::kPerSm;
    return launch_k(norm_kernel<kF32, kV, kRes, kBlock>, dim3(static_cast<unsigned>(need < most ? need : most)),
                    dim3(rows * tpr), 0, stream, pdl, a, tpr, 1.f / a.H);
}

template <bool kF32, bool kRes>
cudaError_t launch_units(const NormArgs &a, int num_sms, cudaStream_t stream, bool pdl)
{
    // 16 columns a thread, fewer where a row would not fill a warp, up to 32
    // to keep its group within 256 threads (several blocks per SM), then 512
    const int units = a.H / Unit<kF32>::kCols;
    constexpr int kFew = kF32 ? 4 : 2;
    int v = kFew;
    while (v > 1 && units / v < 32)
        v /= 2;
    if (units > 256 * v)
        v = 2 * kFew;
    while (units > 512 * v)
        v *= 2;
    const int tpr = ((units + v - 1) / v + 31) / 32 * 32;
    if (v == 1)
        return launch<kF32, 1, kRes, 256>(a, tpr, num_sms, stream, pdl);
    if (v == 2)
        return launch<kF32, 2, kRes, 256>(a, tpr, num_sms, stream, pdl);
    if (kF32 && v == 4)
        return launch<true, 4, kRes, 256>(a, tpr, num_sms, stream, pdl);
    if (v == 2 * kFew)
        return tpr <= 256 ? launch<kF32, 2 * kFew, kRes, 256>(a, tpr, num_sms, stream, pdl)
                          : launch<kF32, 2 * kFew, kRes, 512>(a, tpr, num_sms, stream, pdl);
    return launch<kF32, 4 * kFew, kRes, 512>(a, tpr, num_sms, stream, pdl);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t stream, bool pdl)
{
    if (a.h_f32)
        return a.y ? launch_units<true, true>(a, num_sms, stream, pdl) : launch_units<true, false>(a, num_sms, stream, pdl);
    return a.y ? launch_units<false, true>(a, num_sms, stream, pdl) : launch_units<false, false>(a, num_sms, stream, pdl);
}

}  // namespace moe
