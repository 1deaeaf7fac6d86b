// route_gemm.cu -- the router's logits for more than a few tokens, on the
// tensor cores: logits[t, e] = sum_m x[t, m] w[e, m], bf16 in, fp32 out.
//
// A unit is 128 tokens (MMA M) x kBN experts (MMA N) x one slice of H. The
// output is narrow (T x E with E in the hundreds), so tiles alone would leave
// most SMs idle (64 tiles at T=8192, E=128); a cluster of `slices` CTAs
// shares one tile instead, each over its slice of H, and the partial
// accumulators meet through distributed shared memory: every CTA sends each
// peer the ceil(128 / slices) rows that peer owns, and the owner adds the slices
// in rank order (the same bits whatever the timing) and stores its rows.
//
// Per CTA: warp 0 feeds a ring of TMA stages (128-byte swizzled 64-wide K
// blocks of x and w), warp 1 issues tcgen05.mma, then all 16 warps move the
// accumulators out. The tensor cores truncate as they accumulate, so one long
// chain of MMAs drifts (2.1e-6 of the logits' norm after 128 of them, at
// H=4096 in two slices); the K blocks go round over as many TMEM accumulators
// as fit (four of 64 or 128 experts, two of 192 or 256; 4.7e-7 then), added in
// fp32 on the way out.
#include <cuda_bf16.h>

#include "moe_internal.h"
#include "ptx.cuh"
#include "route_select.cuh"

namespace moe {

namespace {

constexpr int kGemmThreads = 512;
constexpr int kTokens = 128;

template <int kBN>
struct RouteCfg {
    static constexpr int kXBytes = kTokens * 128;
    static constexpr int kStageBytes = kXBytes + kBN * 128;
    static constexpr int kStages = 196608 / kStageBytes;   // 4 at 256 experts to 8 at 64
    static constexpr int kRowFloats = kBN + 4;             // rows of the exchange buffer, 16 bytes apart in banks
    // slices * ceil(128 / slices) rows: at most 133 (seven slices)
    static constexpr int kExchangeBytes = 133 * kRowFloats * 4;
    static constexpr int kDynSmem =
        1024 + (kStages * kStageBytes > kExchangeBytes ? kStages * kStageBytes : kExchangeBytes);
    static constexpr int kAccs = route_accumulators(kBN);
    static constexpr int kTmemCols = kBN <= 64 ? 256 : 512;
    static constexpr uint32_t kIdesc = idesc_bf16_f32(kTokens, kBN);
    static_assert(kAccs * kBN <= kTmemCols, "accumulators");
    static_assert(kBN % 64 == 0 && kBN <= 256, "expert tile");
};

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint32_t *v)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
}

template <int kBN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    route_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ RouteArgs a, int slices, float *__restrict__ logits,
                      uint64_t wait_limit_ns)
{
    using C = RouteCfg<kBN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[C::kStages];
    __shared__ __align__(8) uint64_t bar_empty[C::kStages];
    __shared__ __align__(8) uint64_t bar_done;
    __shared__ uint32_t s_tmem_base;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    volatile int *abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&bar_full[s]), 1);
            mbar_init(smem_u32(&bar_empty[s]), 1);
        }
        mbar_init(smem_u32(&bar_done), 1);
        s_abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w);
    }
    if (warp == 2) {
        tmem_alloc(smem_u32(&s_tmem_base), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem_base;
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a.d_num_tokens, a.T_max);
    const int E = a.E;
    const int rank = static_cast<int>(cluster_ctarank());
    const int n_tiles = (E + kBN - 1) / kBN;
    const int tile = blockIdx.x / slices;
    const int e0 = (tile % n_tiles) * kBN;
    const int t0 = (tile / n_tiles) * kTokens;
    const int blocks = a.H / 64;
    const int kb0 = rank * blocks / slices, kb1 = (rank + 1) * blocks / slices;
    const bool active = t0 < T;     // the same in every CTA of the cluster

    if (active && warp == 0) {
        if (lane == 0) {
            const uint64_t pol_x = l2_policy_evict_first();   // each x row is read by one tile per expert tile
            const uint64_t pol_w = l2_policy_evict_last();
            int issued = 0;
            for (int i = 0; i < kb1 - kb0; ++i) {
                const int s = i % C::kStages;
                const uint32_t phase = (i / C::kStages) & 1;
                if (!mbar_wait_bounded(smem_u32(&bar_empty[s]), phase ^ 1u, abort_flag, wait_limit_ns))
                    break;
                const uint32_t full = smem_u32(&bar_full[s]);
                const uint32_t dst = smem_u32(smem + s * C::kStageBytes);
                mbar_arrive_expect_tx(full, C::kStageBytes);
                tma_load_2d(dst, &tm_x, full, (kb0 + i) * 64, t0, n_tiles == 1 ? pol_x : l2_policy_evict_normal());
                tma_load_2d(dst + C::kXBytes, &tm_w, full, (kb0 + i) * 64, e0, pol_w);
                ++issued;
            }
            // Every load has landed before this CTA's stages become exchange
            // buffers, and before it exits, also if a role gave up (the MMAs
            // otherwise waited for them all).
            for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
                mbar_drain(smem_u32(&bar_full[i % C::kStages]), (i / C::kStages) & 1, wait_limit_ns);
        }
        __syncwarp();
    } else if (active && warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < kb1 - kb0; ++i) {
                const int s = i % C::kStages;
                if (!mbar_wait_bounded(smem_u32(&bar_full[s]), (i / C::kStages) & 1, abort_flag, wait_limit_ns))
                    break;
                tc_fence_after();
                const uint32_t x = smem_u32(smem + s * C::kStageBytes);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_bf16(tmem + (i % C::kAccs) * kBN, smem_desc_kmajor_sw128(x + 32 * k),
                              smem_desc_kmajor_sw128(x + C::kXBytes + 32 * k), C::kIdesc, i >= C::kAccs || k > 0);
                umma_commit(smem_u32(&bar_empty[s]));
            }
            umma_commit(smem_u32(&bar_done));
            // the MMAs issued so far, also after giving up: the accumulators are read and freed below
            mbar_drain(smem_u32(&bar_done), 0, wait_limit_ns);
        }
        __syncwarp();
    }
    if (active) {
        // every MMA and every load of this CTA is complete at the barrier (or its role gave up twice)
        if (lane == 0)
            mbar_wait_bounded(smem_u32(&bar_done), 0, abort_flag, wait_limit_ns);
        __syncwarp();
        tc_fence_after();
        __syncthreads();
        cluster_sync();   // every peer's stages are free: they become the exchange buffers
        // row = TMEM lane; the four warps of a lane quarter take a quarter of its columns each
        const int row = (warp & 3) * 32 + lane;
        const int own = (kTokens + slices - 1) / slices;
        const uint32_t dst = map_to_cta(
            smem_u32(smem) + static_cast<uint32_t>((rank * own + row % own) * C::kRowFloats * 4), row / own);
        const int accs = min(C::kAccs, kb1 - kb0);
#pragma unroll 1
        for (int c = (warp >> 2) * (kBN / 4); c < ((warp >> 2) + 1) * (kBN / 4); c += 16) {
            const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c;
            uint32_t r[C::kAccs][16];
#pragma unroll
            for (int q = 0; q < C::kAccs; ++q)
                if (q < accs)
                    tmem_ld_32x32b_x16(at + q * kBN, r[q]);
            tmem_wait_ld();
#pragma unroll
            for (int q = 1; q < C::kAccs; ++q)
                if (q < accs)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        r[0][i] = __float_as_uint(__uint_as_float(r[0][i]) + __uint_as_float(r[q][i]));
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                st_cluster_v4(dst + (c + i) * 4, r[0] + i);
        }
        cluster_sync();
        const float *const buf = reinterpret_cast<const float *>(smem);
        const int t_own = t0 + rank * own;
        if (!s_abort) {
            const bool whole = E % 4 == 0;   // rows of logits 16-byte aligned
#pragma unroll 4
            for (int i = threadIdx.x; i < own * (kBN / 4); i += kGemmThreads) {
                const int r = i / (kBN / 4), c = 4 * (i % (kBN / 4));
                const float *src = buf + r * C::kRowFloats + c;
                float4 v = *reinterpret_cast<const float4 *>(src);
                for (int s = 1; s < slices; ++s) {
                    const float4 p = *reinterpret_cast<const float4 *>(src + s * own * C::kRowFloats);
                    v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
                }
                if (t_own + r >= T || rank * own + r >= kTokens)
                    continue;
                float *out = logits + static_cast<size_t>(t_own + r) * E + e0 + c;
                if (whole && e0 + c < E) {
                    *reinterpret_cast<float4 *>(out) = v;
                } else if (!whole) {
                    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (e0 + c + j < E)
                            out[j] = f[j];
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (threadIdx.x == 0 && s_abort)
        atomicOr(a.err, MOE_DEVERR_WAIT_TIMEOUT);
}

template <int kBN>
cudaError_t run(const RouteArgs &a, int slices, float *logits, cudaStream_t stream, bool pdl)
{
    using C = RouteCfg<kBN>;
    auto kern = route_gemm_kernel<kBN>;
    static thread_local int attr_done_for_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (attr_done_for_device != dev) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kDynSmem);
        if (e != cudaSuccess)
            return e;
        attr_done_for_device = dev;
    }
    CUtensorMap tm_x, tm_w;
    if (!make_tile_map(&tm_x, a.x, static_cast<uint64_t>(a.T_max), static_cast<uint64_t>(a.H), kTokens) ||
        !make_tile_map(&tm_w, a.w, static_cast<uint64_t>(a.E), static_cast<uint64_t>(a.H), kBN))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(((a.T_max + kTokens - 1) / kTokens) * ((a.E + kBN - 1) / kBN) * slices));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = C::kDynSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(slices);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, tm_x, tm_w, a, slices, logits, kWaitLimitNs);
}

}  // namespace

cudaError_t launch_route_gemm(const RouteArgs &a, float *logits, cudaStream_t stream, bool pdl)
{
    const RouteTile t = route_tile(a.T_max, a.E, a.H);
    switch (t.experts) {
    case 64:
        return run<64>(a, t.slices, logits, stream, pdl);
    case 128:
        return run<128>(a, t.slices, logits, stream, pdl);
    case 192:
        return run<192>(a, t.slices, logits, stream, pdl);
    default:
        return run<256>(a, t.slices, logits, stream, pdl);
    }
}

}  // namespace moe
