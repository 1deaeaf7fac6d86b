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
// order (deterministic: no atomics). T=8192, H=4096 bf16 with dh_add 46.7 us (5.7
// TB/s, 0.86 of the copy rate; 3 us of it the second kernel); T=2047, H=7168 fp32
// 34.4 us (0.89). Up to 16 rows one cluster does it all: T=7, H=7168 6.6 us.
#include "moe_internal.h"
#include "norm_ops.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

// Two sums over the tpr threads (whole warps) of row group `group`, with a
// barrier of the group's own. s: one float2 per warp of the block.
__device__ __forceinline__ float2 row_sums(Pair p, Pair q, int tpr, int group, float2 *s)
{
    const float2 a = halves(p), b = halves(q);
    float u = a.x + a.y, v = b.x + b.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        u += __shfl_xor_sync(0xffffffffu, u, o);
        v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    if (tpr == 32) {
        __syncwarp();
        return make_float2(u, v);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        s[warp] = make_float2(u, v);
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
    const int n = tpr >> 5;      // at most 32
    const float2 w = lane < n ? s[group * n + lane] : make_float2(0.f, 0.f);
    u = w.x;
    v = w.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        u += __shfl_xor_sync(0xffffffffu, u, o);
        v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return make_float2(u, v);
}

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

// The block's row of partial sums out of its row groups' sums s_dw[rows][H],
// in group order.
__device__ __forceinline__ void store_partial(const NormGradArgs &a, const float *s_dw, int rows)
{
    for (int m = threadIdx.x * 4; m < a.H; m += blockDim.x * 4) {
        float4 sum = *reinterpret_cast<const float4 *>(s_dw + m);
        for (int g = 1; g < rows; ++g) {
            const float4 e = *reinterpret_cast<const float4 *>(s_dw + g * a.H + m);
            sum.x += e.x;
            sum.y += e.y;
            sum.z += e.z;
            sum.w += e.w;
        }
        *reinterpret_cast<float4 *>(a.part + static_cast<size_t>(blockIdx.x) * a.H + m) = sum;
    }
}

// Rows of up to 8192 columns, 16 columns a thread. Each row group has a ring of
// `depth` rows in shared memory (h, dx and, where given, dh_add), filled by bulk
// copies that its first thread issues: the barrier of a row's sums also says that
// the row has been taken out of the ring, so the copy of the row `depth` turns on
// starts right behind it. An SM so has up to 200 KB in flight, where loads into
// registers ahead of the barrier held 48 KB (T=8192, H=4096 55 us with those).
constexpr int kStreamThreads = 512;
constexpr int kStreamBytes = 200 * 1024;
constexpr int kMaxDepth = 8;

template <bool kF32, bool kWF32, int kV>
__global__ void __launch_bounds__(kStreamThreads, 1)
    norm_backward_kernel(const __grid_constant__ NormGradArgs a, int tpr, int depth, float inv_H)
{
    using U = Unit<kF32>;
    constexpr int kCols = U::kCols, kPairs = U::kPairs;
    constexpr int kBytes = kF32 ? 4 : 2;
    extern __shared__ __align__(16) uint8_t s_rows[];
    __shared__ __align__(8) uint64_t s_full[16][kMaxDepth];     // of each row group
    __shared__ float2 s_sum[2][kStreamThreads / 32];            // two, so that one barrier a row is enough
    // a thread of the group gave up on this turn's row: written before the barrier of the row's sums, read after it,
    // so that the group leaves together; by turns, since the next row's wait may begin before every thread has read it
    __shared__ int s_abort[16][2];
    const int group = threadIdx.x / tpr, lane = threadIdx.x % tpr;
    const int rows = blockDim.x / tpr;
    if (lane == 0) {
        for (int i = 0; i < depth; ++i)
            mbar_init(smem_u32(&s_full[group][i]), 1);
        s_abort[group][0] = s_abort[group][1] = 0;
    }
    fence_barrier_init();
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a);
    const int step = gridDim.x * rows;
    const int first = blockIdx.x * rows + group;
    const uint32_t h_bytes = a.H * kBytes, dx_bytes = a.H * 2, row_bytes = h_bytes * (a.dh_add ? 2 : 1) + dx_bytes;
    uint8_t *const ring = s_rows + static_cast<size_t>(group) * depth * row_bytes;
    auto copy_row = [&](long long t, int slot) {
        const uint32_t dst = smem_u32(ring + slot * row_bytes), bar = smem_u32(&s_full[group][slot]);
        const uint64_t pol = l2_policy_evict_first();
        mbar_arrive_expect_tx(bar, row_bytes);
        bulk_load(dst, static_cast<const char *>(a.h) + t * a.h_stride * kBytes, h_bytes, bar, pol);
        bulk_load(dst + h_bytes, static_cast<const __nv_bfloat16 *>(a.dx) + t * a.dx_stride, dx_bytes, bar, pol);
        if (a.dh_add)
            bulk_load(dst + h_bytes + dx_bytes, static_cast<const char *>(a.dh_add) + t * a.add_stride * kBytes, h_bytes,
                      bar, pol);
    };
    if (lane == 0)
        for (int i = 0; i < depth && first + static_cast<long long>(i) * step < T; ++i)
            copy_row(first + static_cast<long long>(i) * step, i);
    const int col0 = lane * kCols;
    bool on[kV];
    Weights<kF32, kWF32, kV> w;
    Pair acc[kV][kPairs];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int m = col0 + v * tpr * kCols;
        on[v] = m < a.H;
        if (on[v])
            w.load(a, v, m);
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            acc[v][i] = 0ull;
    }
    int slot = 0, turn = 0;
    uint32_t phase = 0;
    bool gave_up = false;
    for (long long t = first; t < T; t += step, turn ^= 1) {
        volatile int *const abort_flag = &s_abort[group][turn];
        mbar_wait_bounded(smem_u32(&s_full[group][slot]), phase, abort_flag, kWaitLimitNs);
        const uint8_t *const row = ring + slot * row_bytes;
        Pair f[kV][kPairs], g[kV][kPairs], o[kV][kPairs];
        Pair hh = 0ull, qh = 0ull;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int m = col0 + v * tpr * kCols;
            uint4 h = make_uint4(0u, 0u, 0u, 0u), more = h;
            typename U::Half dx = {};
            if (on[v]) {
                h = *reinterpret_cast<const uint4 *>(row + m * kBytes);
                dx = *reinterpret_cast<const typename U::Half *>(row + h_bytes + m * 2);
                if (a.dh_add)
                    more = *reinterpret_cast<const uint4 *>(row + h_bytes + dx_bytes + m * kBytes);
            }
            U::pairs(h, f[v]);
            U::half_pairs(dx, g[v]);
            U::pairs(more, o[v]);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                hh = fma2(f[v][i], f[v][i], hh);
                if (on[v])     // the weights past H were not loaded
                    qh = fma2(w.times(a, v, i, g[v][i]), f[v][i], qh);
            }
        }
        const float2 sums = row_sums(hh, qh, tpr, group, s_sum[turn]);
        if (*abort_flag) {
            gave_up = true;
            break;
        }
        if (lane == 0 && t + static_cast<long long>(depth) * step < T)
            copy_row(t + static_cast<long long>(depth) * step, slot);
        if (++slot == depth) {
            slot = 0;
            phase ^= 1u;
        }
        const float r = rsqrtf(fmaf(sums.x, inv_H, a.eps));
        const float k = -r * r * (sums.y * inv_H);
        const Pair r2 = pair(r, r), k2 = pair(k, k);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            if (!on[v])
                continue;
            const int m = col0 + v * tpr * kCols;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                o[v][i] = fma2(r2, fma2(f[v][i], k2, w.times(a, v, i, g[v][i])), o[v][i]);
                acc[v][i] = fma2(g[v][i], mul2(f[v][i], r2), acc[v][i]);
            }
            U::store(static_cast<char *>(a.dh) + (t * a.out_stride + m) * kBytes, o[v]);
        }
    }
    if (__syncthreads_or(gave_up)) {
        // let the copies in flight land (at most depth of each group), then say so
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
        if (threadIdx.x == 0)
            atomicOr(a.err, MOE_DEVERR_WAIT_TIMEOUT);
        return;
    }
    if (!a.dw)
        return;
    float *const s_dw = reinterpret_cast<float *>(s_rows);      // every row has been taken out
#pragma unroll
    for (int v = 0; v < kV; ++v)
        if (on[v])
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                *reinterpret_cast<float2 *>(s_dw + group * a.H + col0 + v * tpr * kCols + 2 * i) = halves(acc[v][i]);
    __syncthreads();
    store_partial(a, s_dw, rows);
}

// Rows over 8192 columns: one row a block of 1024 threads, 16 or 32 columns and
// 64 registers each, so the weights come out of L1 and dw grows in shared
// memory (T=170, H=12288 bf16 10.6 us in a graph).
template <bool kF32, bool kWF32, int kV>
__global__ void __launch_bounds__(1024, 1) norm_backward_wide_kernel(const __grid_constant__ NormGradArgs a, int tpr,
                                                                     float inv_H)
{
    using U = Unit<kF32>;
    constexpr int kCols = U::kCols, kPairs = U::kPairs;
    constexpr int kBytes = kF32 ? 4 : 2;
    extern __shared__ float4 s_dw4[];
    __shared__ float2 s_sum[2][1024 / 32];
    float *const s_dw = reinterpret_cast<float *>(s_dw4);
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a);
    const int col0 = threadIdx.x * kCols;
    bool on[kV];
    Weights<kF32, kWF32, kV> w;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int m = col0 + v * tpr * kCols;
        on[v] = m < a.H;
        if (on[v])
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                s_dw[m + i] = 0.f;
    }
    int turn = 0;
    for (long long t = blockIdx.x; t < T; t += gridDim.x, turn ^= 1) {
        Pair f[kV][kPairs], g[kV][kPairs];
        Pair hh = 0ull, qh = 0ull;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int m = col0 + v * tpr * kCols;
            uint4 h = make_uint4(0u, 0u, 0u, 0u);
            typename U::Half dx = {};
            if (on[v]) {
                h = ld_stream(static_cast<const char *>(a.h) + (t * a.h_stride + m) * kBytes);
                dx = U::load_half(static_cast<const __nv_bfloat16 *>(a.dx) + t * a.dx_stride + m);
                w.load(a, v, m);
            }
            U::pairs(h, f[v]);
            U::half_pairs(dx, g[v]);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                hh = fma2(f[v][i], f[v][i], hh);
                if (on[v])
                    qh = fma2(w.times(a, v, i, g[v][i]), f[v][i], qh);
            }
        }
        const float2 sums = row_sums(hh, qh, tpr, 0, s_sum[turn]);
        const float r = rsqrtf(fmaf(sums.x, inv_H, a.eps));
        const float k = -r * r * (sums.y * inv_H);
        const Pair r2 = pair(r, r), k2 = pair(k, k);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            if (!on[v])
                continue;
            const int m = col0 + v * tpr * kCols;
            Pair o[kPairs];
            uint4 more = make_uint4(0u, 0u, 0u, 0u);
            if (a.dh_add)
                more = ld_stream(static_cast<const char *>(a.dh_add) + (t * a.add_stride + m) * kBytes);
            U::pairs(more, o);
            w.load(a, v, m);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                o[i] = fma2(r2, fma2(f[v][i], k2, w.times(a, v, i, g[v][i])), o[i]);
                const float2 e = halves(mul2(g[v][i], mul2(f[v][i], r2)));
                s_dw[m + 2 * i] += e.x;
                s_dw[m + 2 * i + 1] += e.y;
            }
            U::store(static_cast<char *>(a.dh) + (t * a.out_stride + m) * kBytes, o);
        }
    }
    if (!a.dw)
        return;
    __syncthreads();
    store_partial(a, s_dw, 1);
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
        if (a.w_f32) {
            const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.w) + m);
            const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.w) + m + 4);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
            w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
        } else {
            const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.w) + m);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[2 * i] = __uint_as_float(x[i] << 16);
                w[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
            }
        }
        if (a.unit_offset)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] += 1.f;
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
    // eight threads a row read the blocks' shares, then add them in a tree
    for (int i = threadIdx.x; i < 8 * kFewRows; i += blockDim.x) {
        const int t = i >> 3;
        const uint32_t b = i & 7;
        float2 s = make_float2(0.f, 0.f);
        if (b < blocks && t < T) {
            uint32_t there;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(there)
                         : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&s_part[t]))), "r"(b));
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(s.x), "=f"(s.y) : "r"(there) : "memory");
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
        }
        if (b == 0) {
            const float r = rsqrtf(fmaf(s.x, inv_H, a.eps));
            s_row[t] = make_float2(r, -r * r * (s.y * inv_H));
        }
    }
    // no block leaves while another may still read its shares: the wait is at the end
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    __syncthreads();
    float acc[8] = {};
#pragma unroll 4
    for (int t = 0; t < (on ? T : 0); ++t) {
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
    if (a.dw && on) {
        store_dw4(a, m, make_float4(acc[0], acc[1], acc[2], acc[3]));
        store_dw4(a, m + 4, make_float4(acc[4], acc[5], acc[6], acc[7]));
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
    int v, tpr, block;
    bool wide;
    int rows() const { return block / tpr; }
    int grid(int T_max) const
    {
        const long long need = (static_cast<long long>(T_max) + rows() - 1) / rows();
        return static_cast<int>(need < 152 ? need : 152);    // a GB300's SMs; the workspace follows it
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
    s.wide = s.tpr > kStreamThreads;
    s.block = s.wide ? s.tpr : kStreamThreads / s.tpr * s.tpr;
    return s;
}

template <bool kF32, bool kWF32, int kV>
cudaError_t run_stream(const NormGradArgs &a, const GradShape &s, cudaStream_t stream)
{
    auto kern = norm_backward_kernel<kF32, kWF32, kV>;
    const int row = a.H * ((a.dh_add ? 2 : 1) * (kF32 ? 4 : 2) + 2);
    int depth = kStreamBytes / (s.rows() * row);
    depth = depth < kMaxDepth ? depth : kMaxDepth;       // two at least: 512 x 16 columns of fp32 are 80 KB a row
    int smem = s.rows() * row * depth;
    const int sums = static_cast<int>(sizeof(float)) * s.rows() * a.H;
    smem = smem > sums ? smem : sums;
    static thread_local int done_for_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (done_for_device != dev) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes)) != cudaSuccess)
            return e;
        done_for_device = dev;
    }
    return launch_k(kern, dim3(s.grid(a.T_max)), dim3(s.block), smem, stream, true, a, s.tpr, depth, 1.f / a.H);
}

template <bool kF32, bool kWF32, int kV>
cudaError_t run_wide(const NormGradArgs &a, const GradShape &s, cudaStream_t stream)
{
    auto kern = norm_backward_wide_kernel<kF32, kWF32, kV>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    if (e != cudaSuccess)
        return e;
    return launch_k(kern, dim3(s.grid(a.T_max)), dim3(s.block), sizeof(float) * a.H, stream, true, a, s.tpr, 1.f / a.H);
}

template <bool kF32, bool kWF32>
cudaError_t run_units(const NormGradArgs &a, const GradShape &s, cudaStream_t stream)
{
    constexpr int kFew = kF32 ? 4 : 2;
    if (s.wide)
        return s.v == kFew ? run_wide<kF32, kWF32, kFew>(a, s, stream) : run_wide<kF32, kWF32, 2 * kFew>(a, s, stream);
    if (s.v == kFew)
        return run_stream<kF32, kWF32, kFew>(a, s, stream);
    if (kF32 && s.v == 2)
        return run_stream<kF32, kWF32, 2>(a, s, stream);
    return run_stream<kF32, kWF32, 1>(a, s, stream);
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
