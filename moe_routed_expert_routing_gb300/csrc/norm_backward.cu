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

// 16 columns a thread in blocks of up to 512 threads, 128 registers each. Rows
// over 8192 columns take 1024 threads of 16 or 32 columns and 64 registers:
// their weights come out of L1 and dw grows in shared memory.
template <int kBlock>
struct GradPlan {
    static constexpr bool kWide = kBlock == 1024;
    static constexpr bool kAhead = !kWide;      // the next row's loads in flight through the barrier
    static constexpr int kPerSm = kBlock == 256 ? 2 : 1;
};

// The norm weights of a thread's columns as they lie in memory (bf16 pairs or
// fp32), so that they stay in registers: read again for every row they cost as
// many load slots as h.
template <bool kF32, bool kWF32, int kV>
struct Weights {
    using U = Unit<kF32>;
    uint32_t raw[kV][kWF32 ? U::kCols : U::kPairs];

    __device__ __forceinline__ void load(const NormGradArgs &a, int v, int m)
    {
        if (!a.w)
            return;
        if constexpr (kWF32) {
#pragma unroll
            for (int i = 0; i < U::kCols; i += 4) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(a.w) + m + i));
                raw[v][i] = u.x;
                raw[v][i + 1] = u.y;
                raw[v][i + 2] = u.z;
                raw[v][i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < U::kCols; i += 4) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.w) + m + i));
                raw[v][i / 2] = u.x;
                raw[v][i / 2 + 1] = u.y;
            }
        }
    }

    // c = the pair i of unit v, times it
    __device__ __forceinline__ Pair times(const NormGradArgs &a, int v, int i, Pair c) const
    {
        if (!a.w)
            return c;
        Pair w;
        if constexpr (kWF32)
            w = pair(__uint_as_float(raw[v][2 * i]), __uint_as_float(raw[v][2 * i + 1]));
        else
            w = widen(raw[v][i]);
        if (a.unit_offset)
            w = add2(w, pair(1.f, 1.f));
        return mul2(c, w);
    }
};

__device__ __forceinline__ int token_count(const NormGradArgs &a)
{
    if (!a.d_num_tokens)
        return a.T_max;
    const int T = *a.d_num_tokens;
    return T < 0 ? 0 : (T > a.T_max ? a.T_max : T);
}

template <bool kF32, bool kWF32, int kV, int kBlock>
__global__ void __launch_bounds__(kBlock, GradPlan<kBlock>::kPerSm)
    norm_backward_kernel(const __grid_constant__ NormGradArgs a, int tpr, float inv_H)
{
    using P = GradPlan<kBlock>;
    using U = Unit<kF32>;
    constexpr int kCols = U::kCols, kPairs = U::kPairs;
    constexpr int kBytes = kF32 ? 4 : 2;
    constexpr bool kAhead = P::kAhead;
    extern __shared__ float4 s_dw4[];           // dw of the block's row groups (kWide: where it grows)
    __shared__ float2 s_sum[2][kBlock / 32];    // two, so that one barrier a row is enough
    float *const s_dw = reinterpret_cast<float *>(s_dw4);
    const int group = threadIdx.x / tpr, lane = threadIdx.x % tpr;
    const int rows = blockDim.x / tpr;
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a);
    const int step = gridDim.x * rows;
    const int col0 = lane * kCols;
    bool on[kV];
    uint4 h[kV], more[kV];
    typename U::Half dx[kV];
    Weights<kF32, kWF32, kV> w;
    Pair acc[P::kWide ? 1 : kV][kPairs];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int m = col0 + v * tpr * kCols;
        on[v] = m < a.H;
        h[v] = more[v] = make_uint4(0u, 0u, 0u, 0u);
        dx[v] = typename U::Half{};
        if (!P::kWide && on[v])
            w.load(a, v, m);
        if constexpr (!P::kWide) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                acc[v][i] = 0ull;
        } else if (on[v]) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                s_dw[m + i] = 0.f;
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
    auto load_more = [&](long long t) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (on[v])
                more[v] = ld_stream(static_cast<const char *>(a.dh_add) +
                                    (t * a.add_stride + col0 + v * tpr * kCols) * kBytes);
    };
    int t = blockIdx.x * rows + group;
    if (kAhead && t < T) {
        load(t);
        if (a.dh_add)
            load_more(t);
    }
    int turn = 0;
    for (int base = blockIdx.x * rows; base < T; base += step, t += step, turn ^= 1) {
        const bool row = t < T;
        if (!kAhead && row) {
            load(t);
            if (a.dh_add)
                load_more(t);
        }
        Pair f[kV][kPairs], g[kV][kPairs];
        Pair hh = 0ull, qh = 0ull;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            U::pairs(h[v], f[v]);
            U::half_pairs(dx[v], g[v]);
        }
        if (kAhead && t + step < T)
            load(t + step);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            if (P::kWide && on[v])
                w.load(a, v, col0 + v * tpr * kCols);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                hh = fma2(f[v][i], f[v][i], hh);
                if (on[v])     // the weights past H were not loaded
                    qh = fma2(w.times(a, v, i, g[v][i]), f[v][i], qh);
            }
        }
        const float2 sums = row_sums(hh, qh, tpr, s_sum[turn]);
        if (!row)
            continue;
        const float r = rsqrtf(fmaf(sums.x, inv_H, a.eps));
        const float k = -r * r * (sums.y * inv_H);
        const Pair r2 = pair(r, r), k2 = pair(k, k);
        Pair o[kV][kPairs];
#pragma unroll
        for (int v = 0; v < kV; ++v)
            U::pairs(more[v], o[v]);       // zero without dh_add
        if (kAhead && a.dh_add && t + step < T)
            load_more(t + step);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            if (!on[v])
                continue;
            const int m = col0 + v * tpr * kCols;
            if (P::kWide)
                w.load(a, v, m);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                o[v][i] = fma2(r2, fma2(f[v][i], k2, w.times(a, v, i, g[v][i])), o[v][i]);
                const Pair n = mul2(f[v][i], r2);
                if constexpr (P::kWide) {
                    const float2 e = halves(mul2(g[v][i], n));
                    s_dw[m + 2 * i] += e.x;
                    s_dw[m + 2 * i + 1] += e.y;
                } else {
                    acc[v][i] = fma2(g[v][i], n, acc[v][i]);
                }
            }
            U::store(static_cast<char *>(a.dh) + (t * a.out_stride + m) * kBytes, o[v]);
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

__device__ __forceinline__ void store_dw4(const NormGradArgs &a, int m, const float4 &v)
{
    if (a.w_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(a.dw) + m) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.dw) + m) =
            make_uint2(narrow(pair(v.x, v.y)), narrow(pair(v.z, v.w)));
}

// dw[m] = sum of the n partial rows: a block takes 16 x 4 columns, 32 threads
// of each every 32nd row, then their sums in order.
constexpr int kSumThreads = 512;

__global__ void __launch_bounds__(kSumThreads) norm_dw_kernel(const __grid_constant__ NormGradArgs a, int n)
{
    constexpr int kWays = kSumThreads / 16;
    __shared__ float4 s[kWays][16];
    const int way = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int m = (blockIdx.x * 16 + lane) * 4;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    pdl_wait();
    pdl_trigger();
    const float *const p = a.part + m;     // H is a multiple of 64
#pragma unroll 5
    for (int i = way; i < n; i += kWays) {
        const float4 e = *reinterpret_cast<const float4 *>(p + static_cast<size_t>(i) * a.H);
        sum.x += e.x;
        sum.y += e.y;
        sum.z += e.z;
        sum.w += e.w;
    }
    s[way][lane] = sum;
    __syncthreads();
    if (way)
        return;
    for (int i = 1; i < kWays; ++i) {
        const float4 e = s[i][lane];
        sum.x += e.x;
        sum.y += e.y;
        sum.z += e.z;
        sum.w += e.w;
    }
    store_dw4(a, m, sum);
}

// Up to kFewRows rows: one cluster of up to 8 blocks, each with its share of
// the columns of every row, so that dw needs no partial rows and no second
// kernel. The rows' sums go round the cluster in shared memory; a row's
// columns are read again after that, out of L1.
constexpr int kFewRows = 16;
constexpr int kFewThreads = 512;

template <bool kF32>
__global__ void __launch_bounds__(kFewThreads) norm_backward_few_kernel(const __grid_constant__ NormGradArgs a,
                                                                        float inv_H)
{
    constexpr int kBytes = kF32 ? 4 : 2;
    constexpr int kVecs = kF32 ? 2 : 1;          // 16-byte words of a thread's 8 columns
    __shared__ float2 s_warp[kFewRows][kFewThreads / 32];
    __shared__ float2 s_part[kFewRows];          // this block's share of each row's sums
    __shared__ float2 s_row[kFewRows];           // r and -r^2 mean(q h)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    uint32_t rank, blocks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(blocks));
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a);
    const int m = 8 * static_cast<int>(rank * blockDim.x + threadIdx.x);
    const bool on = m < a.H;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = 1.f;
    if (a.w && on) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = (a.w_f32 ? static_cast<const float *>(a.w)[m + i]
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.w)[m + i])) +
                   (a.unit_offset ? 1.f : 0.f);
    }
    // the 8 columns of row t of an h-typed tensor, and of dx
    auto row8 = [&](const void *base, long long stride, int t, float(&f)[8]) {
        const char *const p = static_cast<const char *>(base) + (t * stride + m) * kBytes;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p + 16 * v);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kF32) {
                    f[4 * v + i] = __uint_as_float(x[i]);
                } else {
                    f[2 * i] = __uint_as_float(x[i] << 16);
                    f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
                }
            }
        }
    };
    auto dx8 = [&](int t, float(&f)[8]) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.dx) + t * a.dx_stride + m);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(x[i] << 16);
            f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
    };
#pragma unroll 8
    for (int t = 0; t < T; ++t) {
        float hh = 0.f, qh = 0.f;
        if (on) {
            float f[8], g[8];
            row8(a.h, a.h_stride, t, f);
            dx8(t, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                hh = fmaf(f[i], f[i], hh);
                qh = fmaf(g[i] * w[i], f[i], qh);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            hh += __shfl_xor_sync(0xffffffffu, hh, o);
            qh += __shfl_xor_sync(0xffffffffu, qh, o);
        }
        if (lane == 0)
            s_warp[t][warp] = make_float2(hh, qh);
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < T) {
        float2 s = s_warp[threadIdx.x][0];
        for (int i = 1; i < warps; ++i) {
            s.x += s_warp[threadIdx.x][i].x;
            s.y += s_warp[threadIdx.x][i].y;
        }
        s_part[threadIdx.x] = s;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (static_cast<int>(threadIdx.x) < T) {
        float2 s = make_float2(0.f, 0.f);
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&s_part[threadIdx.x]));
        for (uint32_t b = 0; b < blocks; ++b) {
            uint32_t there;
            float2 e;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(b));
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(e.x), "=f"(e.y) : "r"(there) : "memory");
            s.x += e.x;
            s.y += e.y;
        }
        const float r = rsqrtf(fmaf(s.x, inv_H, a.eps));
        s_row[threadIdx.x] = make_float2(r, -r * r * (s.y * inv_H));
    }
    // no block leaves, or writes dh (which may be h), while another still reads its sums
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();
    if (!on)
        return;
    float acc[8] = {};
#pragma unroll 4
    for (int t = 0; t < T; ++t) {
        float f[8], g[8], o[8] = {};
        row8(a.h, a.h_stride, t, f);
        dx8(t, g);
        if (a.dh_add)
            row8(a.dh_add, a.add_stride, t, o);
        const float2 rk = s_row[t];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = fmaf(rk.x, fmaf(f[i], rk.y, g[i] * w[i]), o[i]);
            acc[i] = fmaf(g[i], f[i] * rk.x, acc[i]);
        }
        char *const p = static_cast<char *>(a.dh) + (t * a.out_stride + m) * kBytes;
        if constexpr (kF32) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
        } else {
            *reinterpret_cast<uint4 *>(p) = make_uint4(narrow(pair(o[0], o[1])), narrow(pair(o[2], o[3])),
                                                       narrow(pair(o[4], o[5])), narrow(pair(o[6], o[7])));
        }
    }
    if (a.dw) {
        store_dw4(a, m, make_float4(acc[0], acc[1], acc[2], acc[3]));
        store_dw4(a, m + 4, make_float4(acc[4], acc[5], acc[6], acc[7]));
    }
}

template <bool kF32>
cudaError_t run_few(const NormGradArgs &a, cudaStream_t stream)
{
    // 128 threads a block (8 columns each) while 8 blocks hold the row, more beyond
    const int units = a.H / 8;
    int blocks = 1;
    while (blocks < 8 && units > 128 * blocks)
        blocks *= 2;
    const int threads = ((units + blocks - 1) / blocks + 31) / 32 * 32;     // at most 512: H <= 32768
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, norm_backward_few_kernel<kF32>, a, 1.f / a.H);
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

template <bool kF32, bool kWF32, int kV, int kBlock>
cudaError_t run(const NormGradArgs &a, const GradShape &s, cudaStream_t stream)
{
    auto kern = norm_backward_kernel<kF32, kWF32, kV, kBlock>;
    const size_t smem = a.dw || GradPlan<kBlock>::kWide ? sizeof(float) * s.rows() * a.H : 0;
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
        if (e != cudaSuccess)
            return e;
    }
    return launch_k(kern, dim3(s.grid(a.T_max)), dim3(s.block), smem, stream, true, a, s.tpr, 1.f / a.H);
}

template <bool kF32, bool kWF32>
cudaError_t run_units(const NormGradArgs &a, const GradShape &s, cudaStream_t stream)
{
    constexpr int kFew = kF32 ? 4 : 2;
    if (s.v == 2 * kFew)
        return run<kF32, kWF32, 2 * kFew, 1024>(a, s, stream);
    if (s.v == kFew)
        return s.tpr <= 256 ? run<kF32, kWF32, kFew, 256>(a, s, stream)
                            : (s.tpr <= 512 ? run<kF32, kWF32, kFew, 512>(a, s, stream)
                                            : run<kF32, kWF32, kFew, 1024>(a, s, stream));
    if (kF32 && s.v == 2)
        return run<kF32, kWF32, 2, 256>(a, s, stream);
    return run<kF32, kWF32, 1, 256>(a, s, stream);
}

}  // namespace

int norm_grad_part_rows(int T_max, int H, bool h_f32)
{
    return T_max <= kFewRows ? 0 : grad_shape(H, h_f32).grid(T_max);
}

cudaError_t launch_norm_backward(const NormGradArgs &a, cudaStream_t stream)
{
    if (a.T_max <= kFewRows)
        return a.h_f32 ? run_few<true>(a, stream) : run_few<false>(a, stream);
    const GradShape s = grad_shape(a.H, a.h_f32);
    const cudaError_t e = a.h_f32 ? (a.w_f32 ? run_units<true, true>(a, s, stream) : run_units<true, false>(a, s, stream))
                                  : (a.w_f32 ? run_units<false, true>(a, s, stream) : run_units<false, false>(a, s, stream));
    if (e != cudaSuccess || !a.dw)
        return e;
    return launch_k(norm_dw_kernel, dim3(a.H / 64), dim3(kSumThreads), 0, stream, true, a, s.grid(a.T_max));
}

}  // namespace moe
