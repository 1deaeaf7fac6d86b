// expert_backward.cu -- gradients of the experts' MLP on a batch sorted by
// expert, and the grouped products they (and the router's gradient) are made
// of, on tcgen05/TMEM CTA pairs.
//
// With g, u = x W13^T (gate and up halves), s = sigmoid(g), a = g s u:
//   da = dy W2,   du = da g s,   dg = da u s (1 + g (1 - s))
//   dx = [dg du] W13,   dW2[e] = dy^T a,   dW13[e] = [dg du]^T x
// with the sums of the last two over expert e's rows. g and u are computed
// again: the forward keeps neither, and they are a quarter of the products.
//
// Two kernels:
//  * act_grad_kernel -- a tile of 256 rows x 128 columns of the intermediate
//    size holds g, u and da together in TMEM (384 of its 512 columns), so the
//    three meet in registers in fp32 and only a and [dg du] are stored, each
//    rounded to bf16 once: the operands of the products that follow;
//  * products_kernel -- dx, dW13 and dW2 as the units of one persistent grid.
//
// Operand placement. A CTA pair multiplies 256 x 256 tiles (M=256, N=256,
// cta_group::2), each CTA holding half of A and half of B. Operands whose K
// runs along memory rows (x, dy, [dg du] as dx's A) are K-major tiles; those
// whose K runs across rows (W2 and W13 as B of da and dx, both operands of the
// weight gradients) are read as they lie, as MN-major tiles of 64 K rows x 64
// columns with 128-byte swizzling: no operand is transposed in memory. Both
// kinds fill the same 16 KB half stages, so one ring serves every unit.
//
// Rows behind an expert's last one. As M rows they are multiplied and not
// stored. As K rows (weight gradients) they must not count: the last K block
// of an expert with rows % 64 != 0 lands on a barrier of the CTA's own, one
// warp zeroes the rows up to the next multiple of 16 in both operands (they
// may hold another expert's rows or, past the valid ones, anything), and the
// MMAs beyond that multiple are not issued.
#include <cuda_bf16.h>

#include "moe_internal.h"
#include "ptx.cuh"
#include "tiles.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kBK = 64;                      // K elements of a stage
constexpr int kUmmaK = 16;
constexpr int kTileRows = 256;               // rows of a CTA pair's tile
constexpr int kHalf = 128 * 128;             // bytes of one operand's half tile: 128 x 64 bf16
constexpr int kAtom = 64 * 128;              // bytes of an MN-major block: 64 K rows x 64 columns
constexpr int kStageBytes = 2 * kHalf;
constexpr int kStages = 6;
constexpr int kScratch = 4 * 32 * 36 * 4;    // a 32 x 36-word transpose scratch per epilogue warp
constexpr int kDynSmem = 1024 + kStages * kStageBytes + kScratch;
constexpr uint32_t kMajorA = 1u << 15, kMajorB = 1u << 16;   // instruction descriptor: operand is MN-major

// Shared-memory descriptor of an MN-major bf16 tile: blocks of 64 K rows x 64
// columns (128-byte rows, 128-byte swizzle), 8 K rows every 1024 bytes
// (stride offset), the next 64 columns one block on (leading offset). A K step
// of 16 is 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mnmajor_sw128(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(kAtom >> 4) << 16 |
           static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}

__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void fence_proxy_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// What every thread of a CTA pair's kernel starts from.
struct PairState {
    uint8_t *smem;          // stages, 1024-byte aligned
    uint32_t tmem;
    uint32_t rank;
    int cluster, clusters;
};

struct PairBars {
    uint64_t full[kStages];    // used in CTA 0: one arrival and the bytes of each CTA
    uint64_t empty[kStages];
    uint64_t tail[kStages];    // a K block whose rows one warp zeroes before it counts as full
    uint64_t tfull[2];
    uint64_t tempty[2];        // used in CTA 0
    uint64_t drain;            // used in CTA 0
};

// Barriers, TMEM, the experts' offsets (clamped to the batch) and their row tiles.
__device__ __forceinline__ PairState pair_begin(uint8_t *smem_raw, PairBars &bars, uint32_t &s_tmem, int &s_abort,
                                                int *s_off, int *s_tp, const int32_t *offsets, int E, int cap)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    PairState st;
    st.smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    st.rank = cluster_ctarank();
    st.cluster = blockIdx.x >> 1;
    st.clusters = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 2);
            mbar_init(smem_u32(&bars.empty[s]), 1);
            mbar_init(smem_u32(&bars.tail[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bars.tfull[b]), 1);
            mbar_init(smem_u32(&bars.tempty[b]), 8);   // 4 epilogue warps x 2 CTAs
        }
        mbar_init(smem_u32(&bars.drain), 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        tmem_alloc_pair(smem_u32(&s_tmem), 512);
        tmem_relinquish_pair();
    }
    for (int i = threadIdx.x; i <= E; i += kThreads) {
        const int o = offsets[i];
        s_off[i] = o < 0 ? 0 : (o > cap ? cap : o);
    }
    __syncthreads();
    if (warp == 3)
        build_tile_prefix(s_off, s_tp, E, kTileRows, lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers initialised before any remote arrive
    tc_fence_after();
    st.tmem = s_tmem;
    return st;
}

__device__ __forceinline__ void pair_end(const PairState &st, int &s_abort, int32_t *err)
{
    tc_fence_before();
    __syncthreads();
    if (s_abort) {
        // give-up path: let loads and remote arrivals still in flight land first
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
    cluster_sync();   // neither CTA leaves while its peer may still touch its shared memory
    if ((threadIdx.x >> 5) == 2) {
        tc_fence_after();
        tmem_dealloc_pair(st.tmem, 512);
    }
    if (threadIdx.x == 0 && s_abort)
        atomicOr(err, MOE_DEVERR_WAIT_TIMEOUT);
}

struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// ------------------------------------------------------------------ a and [dg du]

struct ActArgs {
    CUtensorMap x, dy;       // [cap, H], boxes of 64 x 128 rows
    CUtensorMap w13;         // [E * 2I, H], boxes of 64 x 128 rows
    CUtensorMap w2;          // [E * H, I], boxes of 64 x 64 rows
    const int32_t *offsets;
    int32_t *err;
    __nv_bfloat16 *act;      // [cap, I]
    __nv_bfloat16 *dgu;      // [cap, 2I]
    uint64_t wait_limit_ns;
    int E, cap, H, I;
};

struct ActUnit {
    int e, row0, rows, n0;
};

// Column tile, then row tile: the row tiles that share one weight tile go to
// neighbouring pairs.
__device__ __forceinline__ ActUnit act_unit(int u, const int *s_off, const int *s_tp, int E, int NT)
{
    ActUnit t;
    t.e = find_expert(s_tp, E, u, NT);
    const int local = u - s_tp[t.e] * NT;
    const int tiles = s_tp[t.e + 1] - s_tp[t.e];
    const int nt = local / tiles;
    t.row0 = s_off[t.e] + (local - nt * tiles) * kTileRows;
    t.rows = min(s_off[t.e + 1] - t.row0, kTileRows);
    t.n0 = nt * 128;
    return t;
}

// One element's gradients from its gate, up and da values.
__device__ __forceinline__ void swiglu_grad(float g, float u, float d, float &a, float &dg, float &du)
{
    const float s = 1.0f / (1.0f + expf(-g));
    const float silu = g * s;
    a = silu * u;
    du = d * silu;
    dg = d * u * (s * (1.0f + g * (1.0f - s)));
}

// TMEM columns: da of even and odd units in 0..127 and 128..255, gate and up
// in 256..511. A unit's da comes first, so that it can be multiplied while the
// unit before is still being read out: a third of the unit's MMAs, which hides
// that unit's epilogue.
__global__ void __launch_bounds__(kThreads, 1) act_grad_kernel(const __grid_constant__ ActArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) PairBars bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_off[kMaxExperts + 1];
    __shared__ int s_tp[kMaxExperts + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PairState st = pair_begin(smem_raw, bars, s_tmem, s_abort, s_off, s_tp, args.offsets, args.E, args.cap);
    volatile int *abort_flag = &s_abort;
    const int NT = (args.I + 127) / 128;
    const int units = s_tp[args.E] * NT;
    const int k_blocks = args.H / kBK;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_w = l2_policy_evict_normal();
            const uint64_t pol_a = l2_policy_evict_last();
            Ring r;
            bool ok = true;
            for (int u = st.cluster; ok && u < units; u += st.clusters) {
                const ActUnit t = act_unit(u, s_off, s_tp, args.E, NT);
                const int a_row = t.row0 + 128 * static_cast<int>(st.rank);
                const int w2_row = t.e * args.H;
                const int w13_row = t.e * 2 * args.I + (st.rank ? args.I : 0) + t.n0;
                for (int kb = 0; kb < 2 * k_blocks; ++kb, r.next()) {
                    if (!mbar_wait_bounded(smem_u32(&bars.empty[r.stage]), r.phase ^ 1u, abort_flag,
                                           args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = map_to_cta(smem_u32(&bars.full[r.stage]), 0);
                    const uint32_t a_dst = smem_u32(st.smem + r.stage * kStageBytes);
                    const uint32_t b_dst = a_dst + kHalf;
                    if (kb < k_blocks) {
                        mbar_arrive_expect_tx_cluster(full, kHalf + kAtom);
                        tma_load_2d_pair(a_dst, &args.dy, full, kb * kBK, a_row, pol_a);
                        tma_load_2d_pair(b_dst, &args.w2, full, t.n0 + 64 * static_cast<int>(st.rank),
                                         w2_row + kb * kBK, pol_w);
                    } else {
                        mbar_arrive_expect_tx_cluster(full, kStageBytes);
                        tma_load_2d_pair(a_dst, &args.x, full, (kb - k_blocks) * kBK, a_row, pol_a);
                        tma_load_2d_pair(b_dst, &args.w13, full, (kb - k_blocks) * kBK, w13_row, pol_w);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && st.rank == 0) {
            constexpr uint32_t kIdescDa = idesc_bf16_f32(256, 128) | kMajorB;
            constexpr uint32_t kIdescGu = idesc_bf16_f32(256, 256);
            Ring r;
            bool ok = true;
            int local = 0;
            for (int u = st.cluster; ok && u < units; u += st.clusters, ++local) {
                for (int kb = 0; kb < 2 * k_blocks; ++kb, r.next()) {
                    const bool da = kb < k_blocks;
                    if (kb == k_blocks) {
                        // gate and up of the unit before have been read (and with them the da before that)
                        if (!mbar_wait_bounded(smem_u32(&bars.tempty[0]), (local & 1) ^ 1u, abort_flag,
                                               args.wait_limit_ns)) {
                            ok = false;
                            break;
                        }
                    }
                    if (!mbar_wait_bounded(smem_u32(&bars.full[r.stage]), r.phase, abort_flag, args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(st.smem + r.stage * kStageBytes);
                    const uint32_t b_addr = a_addr + kHalf;
                    const uint32_t d = st.tmem + (da ? 128 * (local & 1) : 256);
                    const bool first = kb == 0 || kb == k_blocks;
#pragma unroll
                    for (int kk = 0; kk < kBK / kUmmaK; ++kk) {
                        const uint64_t b_desc = da ? smem_desc_mnmajor_sw128(b_addr + kk * 2048)
                                                   : smem_desc_kmajor_sw128(b_addr + kk * 32);
                        umma_bf16_pair(d, smem_desc_kmajor_sw128(a_addr + kk * 32), b_desc, da ? kIdescDa : kIdescGu,
                                       (first && kk == 0) ? 0u : 1u);
                    }
                    umma_commit_pair(smem_u32(&bars.empty[r.stage]), 0x3);
                }
                if (ok)
                    umma_commit_pair(smem_u32(&bars.tfull[0]), 0x3);
            }
            umma_commit_pair(smem_u32(&bars.drain), 0x1);
            mbar_drain(smem_u32(&bars.drain), 0, args.wait_limit_ns);
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int q = warp - 4;
        int local = 0;
        for (int u = st.cluster; u < units; u += st.clusters, ++local) {
            const ActUnit t = act_unit(u, s_off, s_tp, args.E, NT);
            int ok = 0;
            if (lane == 0)
                ok = mbar_wait_bounded(smem_u32(&bars.tfull[0]), local & 1, abort_flag, args.wait_limit_ns) ? 1 : 0;
            if (!__shfl_sync(kFull, ok, 0))
                break;
            tc_fence_after();
            const uint32_t lanes = st.tmem + (static_cast<uint32_t>(q * 32) << 16);
            const uint32_t t_da = lanes + 128 * (local & 1), t_gu = lanes + 256;
            const int r = 128 * static_cast<int>(st.rank) + q * 32 + lane;
            const bool valid = r < t.rows;
            const size_t row = static_cast<size_t>(t.row0 + r);
            __nv_bfloat16 *const act = args.act + row * args.I + t.n0;
            __nv_bfloat16 *const dg = args.dgu + row * 2 * args.I + t.n0;
            __nv_bfloat16 *const du = dg + args.I;
            const int cols = args.I - t.n0;
#pragma unroll 1
            for (int c = 0; c < 128 && c < cols; c += 16) {
                uint32_t vg[16], vu[16], vd[16];
                tmem_ld_32x32b_x16(t_gu + c, vg);
                tmem_ld_32x32b_x16(t_gu + 128 + c, vu);
                tmem_ld_32x32b_x16(t_da + c, vd);
                tmem_wait_ld();
                uint32_t oa[8], og[8], ou[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float a[2], g[2], w[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        swiglu_grad(__uint_as_float(vg[2 * i + j]), __uint_as_float(vu[2 * i + j]),
                                    __uint_as_float(vd[2 * i + j]), a[j], g[j], w[j]);
                    oa[i] = pack_bf16x2(a[0], a[1]);
                    og[i] = pack_bf16x2(g[0], g[1]);
                    ou[i] = pack_bf16x2(w[0], w[1]);
                }
                if (valid) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        reinterpret_cast<uint4 *>(act + c)[i] = make_uint4(oa[4 * i], oa[4 * i + 1], oa[4 * i + 2], oa[4 * i + 3]);
                        reinterpret_cast<uint4 *>(dg + c)[i] = make_uint4(og[4 * i], og[4 * i + 1], og[4 * i + 2], og[4 * i + 3]);
                        reinterpret_cast<uint4 *>(du + c)[i] = make_uint4(ou[4 * i], ou[4 * i + 1], ou[4 * i + 2], ou[4 * i + 3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(map_to_cta(smem_u32(&bars.tempty[0]), 0));
        }
    }
    pair_end(st, s_abort, args.err);
}

// ------------------------------------------------------------------ products

struct ProductUnit {
    int job, e;
    int m0, rows;        // first output row (rows kind: of the sorted batch) and how many of the 256 there are
    int n0;
    int k_blocks, rem;   // K blocks of one part; rows of its last block when that is not whole, else 0
    int k_row0;          // weights kind: first K row
};

struct ProductArgs {
    ProductJob job[3];
    CUtensorMap map[6];      // A and B of each job
    const int32_t *offsets;
    int32_t *err;
    uint64_t wait_limit_ns;
    int jobs, E, cap;
};

__device__ __forceinline__ int job_units(const ProductJob &j, const int *s_tp, int E)
{
    const int NT = (j.N + 255) / 256;
    return j.by_rows ? s_tp[E] * NT : E * ((j.M + 255) / 256) * NT;
}

__device__ __forceinline__ ProductUnit product_unit(int u, const ProductArgs &args, const int *s_off, const int *s_tp)
{
    ProductUnit t;
    t.job = 0;
    for (; t.job + 1 < args.jobs; ++t.job) {
        const int n = job_units(args.job[t.job], s_tp, args.E);
        if (u < n)
            break;
        u -= n;
    }
    const ProductJob &j = args.job[t.job];
    const int NT = (j.N + 255) / 256;
    if (j.by_rows) {
        const int rt = u / NT;
        t.n0 = (u - rt * NT) * 256;
        t.e = find_expert(s_tp, args.E, rt, 1);
        t.m0 = s_off[t.e] + (rt - s_tp[t.e]) * kTileRows;
        t.rows = min(s_off[t.e + 1] - t.m0, kTileRows);
        t.k_blocks = j.k_blocks;
        t.rem = 0;
        t.k_row0 = 0;
    } else {
        const int MT = (j.M + 255) / 256;
        t.e = u / (MT * NT);
        u -= t.e * MT * NT;
        const int mt = u / NT;
        t.m0 = mt * 256;
        t.n0 = (u - mt * NT) * 256;
        t.rows = min(j.M - t.m0, 256);
        const int k = max(s_off[t.e + 1] - s_off[t.e], 0);
        t.k_blocks = (k + kBK - 1) / kBK;
        t.rem = k % kBK;
        t.k_row0 = s_off[t.e];
    }
    return t;
}

// Rows m0 + 128 rank + 32 q .. + 31 of a tile out of TMEM (or zeros) into
// [*, ld] memory at `base` + row * ld + n0. Through shared memory, so that 8
// lanes store 128 whole bytes of one row.
__device__ __forceinline__ void store_rows(uint32_t t_row, float *scratch, const ProductJob &j, size_t base, int first,
                                           int rows, int n0, bool zero)
{
    const int lane = threadIdx.x & 31;
    const int cols = min(j.N - n0, 256);     // a multiple of 64
    uint4 *const mine = reinterpret_cast<uint4 *>(scratch + lane * 36);
    const int step = j.out_f32 ? 32 : 64;
#pragma unroll 1
    for (int c = 0; c < cols; c += step) {
        uint32_t d[32];
        if (zero) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                d[i] = 0u;
        } else if (j.out_f32) {
            tmem_ld_32x32b_x32(t_row + c, d);
            tmem_wait_ld();
        } else {
            uint32_t v[32];
            tmem_ld_32x32b_x32(t_row + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                d[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            tmem_ld_32x32b_x32(t_row + c + 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                d[16 + i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mine[i] = make_uint4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int rr = 4 * it + (lane >> 3);
            uint4 v = *reinterpret_cast<const uint4 *>(scratch + rr * 36 + (lane & 7) * 4);
            if (first + rr < rows) {
                const size_t o = base + static_cast<size_t>(first + rr) * j.ld + n0 + c + (lane & 7) * (step / 8);
                if (j.out_f32) {
                    float4 *const p = reinterpret_cast<float4 *>(static_cast<float *>(j.out) + o);
                    float4 f = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                                           __uint_as_float(v.w));
                    if (j.accumulate) {
                        const float4 old = *p;
                        f.x += old.x;
                        f.y += old.y;
                        f.z += old.z;
                        f.w += old.w;
                    }
                    *p = f;
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(j.out) + o) = v;
                }
            }
        }
        __syncwarp();
    }
}

__global__ void __launch_bounds__(kThreads, 1) products_kernel(const __grid_constant__ ProductArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) PairBars bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_off[kMaxExperts + 1];
    __shared__ int s_tp[kMaxExperts + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PairState st = pair_begin(smem_raw, bars, s_tmem, s_abort, s_off, s_tp, args.offsets, args.E, args.cap);
    volatile int *abort_flag = &s_abort;
    int units = 0;
    for (int j = 0; j < args.jobs; ++j)
        units += job_units(args.job[j], s_tp, args.E);

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = l2_policy_evict_normal();
            const int half = 128 * static_cast<int>(st.rank);
            Ring r;
            bool ok = true;
            for (int u = st.cluster; ok && u < units; u += st.clusters) {
                const ProductUnit t = product_unit(u, args, s_off, s_tp);
                const ProductJob &j = args.job[t.job];
                const CUtensorMap *ma = &args.map[2 * t.job], *mb = ma + 1;
                const int total = t.k_blocks * (j.by_rows ? 1 : j.parts);
                int part = 0, kp = 0;     // weights kind: the part, and the K block inside it; rows kind: kp mod wrap
                const int period = j.by_rows ? j.wrap : t.k_blocks;
                for (int kb = 0; kb < total; ++kb, r.next()) {
                    if (!mbar_wait_bounded(smem_u32(&bars.empty[r.stage]), r.phase ^ 1u, abort_flag,
                                           args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = map_to_cta(smem_u32(&bars.full[r.stage]), 0);
                    const uint32_t a_dst = smem_u32(st.smem + r.stage * kStageBytes);
                    const uint32_t b_dst = a_dst + kHalf;
                    if (j.by_rows) {
                        const int b_row = t.e * j.b_expert_rows + kp * kBK;
                        mbar_arrive_expect_tx_cluster(full, kStageBytes);
                        tma_load_2d_pair(a_dst, ma, full, kb * kBK, t.m0 + half, pol);
                        tma_load_2d_pair(b_dst, mb, full, t.n0 + half, b_row, pol);
                        tma_load_2d_pair(b_dst + kAtom, mb, full, t.n0 + half + 64, b_row, pol);
                    } else {
                        const int a_col = t.m0 + half + part * j.part_cols;
                        const int row = t.k_row0 + kp * kBK;
                        if (t.rem && kp + 1 == t.k_blocks) {
                            const uint32_t tail = smem_u32(&bars.tail[r.stage]);
                            mbar_arrive_expect_tx(tail, kStageBytes);
                            tma_load_2d(a_dst, ma, tail, a_col, row, pol);
                            tma_load_2d(a_dst + kAtom, ma, tail, a_col + 64, row, pol);
                            tma_load_2d(b_dst, mb, tail, t.n0 + half, row, pol);
                            tma_load_2d(b_dst + kAtom, mb, tail, t.n0 + half + 64, row, pol);
                        } else {
                            mbar_arrive_expect_tx_cluster(full, kStageBytes);
                            tma_load_2d_pair(a_dst, ma, full, a_col, row, pol);
                            tma_load_2d_pair(a_dst + kAtom, ma, full, a_col + 64, row, pol);
                            tma_load_2d_pair(b_dst, mb, full, t.n0 + half, row, pol);
                            tma_load_2d_pair(b_dst + kAtom, mb, full, t.n0 + half + 64, row, pol);
                        }
                    }
                    if (++kp == period) {
                        kp = 0;
                        ++part;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && st.rank == 0) {
            Ring r;
            bool ok = true;
            int local = 0;
            for (int u = st.cluster; ok && u < units; u += st.clusters, ++local) {
                const ProductUnit t = product_unit(u, args, s_off, s_tp);
                const ProductJob &j = args.job[t.job];
                const int total = t.k_blocks * (j.by_rows ? 1 : j.parts);
                const uint32_t idesc = idesc_bf16_f32(256, 256) | kMajorB | (j.by_rows ? 0u : kMajorA);
                const int buf = local & 1;
                if (!mbar_wait_bounded(smem_u32(&bars.tempty[buf]), ((local >> 1) & 1) ^ 1u, abort_flag,
                                       args.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = st.tmem + buf * 256;
                int kp = 0;
                for (int kb = 0; kb < total; ++kb, r.next()) {
                    if (!mbar_wait_bounded(smem_u32(&bars.full[r.stage]), r.phase, abort_flag, args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(st.smem + r.stage * kStageBytes);
                    const uint32_t b_addr = a_addr + kHalf;
                    const bool last = ++kp == t.k_blocks;
                    if (last)
                        kp = 0;
                    const int steps = (last && t.rem) ? (t.rem + kUmmaK - 1) / kUmmaK : kBK / kUmmaK;
#pragma unroll
                    for (int kk = 0; kk < kBK / kUmmaK; ++kk)
                        if (kk < steps) {
                            const uint64_t a_desc = j.by_rows ? smem_desc_kmajor_sw128(a_addr + kk * 32)
                                                              : smem_desc_mnmajor_sw128(a_addr + kk * 2048);
                            umma_bf16_pair(d, a_desc, smem_desc_mnmajor_sw128(b_addr + kk * 2048), idesc,
                                           (kb > 0 || kk > 0) ? 1u : 0u);
                        }
                    umma_commit_pair(smem_u32(&bars.empty[r.stage]), 0x3);
                }
                if (ok)
                    umma_commit_pair(smem_u32(&bars.tfull[buf]), 0x3);
            }
            umma_commit_pair(smem_u32(&bars.drain), 0x1);
            mbar_drain(smem_u32(&bars.drain), 0, args.wait_limit_ns);
        }
        __syncwarp();
    } else if (warp == 3) {
        // the rows of a partial last K block that no longer belong to the expert
        Ring r;
        uint32_t parity = 0;      // of each stage's tail barrier
        bool ok = true;
        for (int u = st.cluster; ok && u < units; u += st.clusters) {
            const ProductUnit t = product_unit(u, args, s_off, s_tp);
            const ProductJob &j = args.job[t.job];
            const int total = t.k_blocks * (j.by_rows ? 1 : j.parts);
            int kp = 0;
            for (int kb = 0; ok && kb < total; ++kb, r.next()) {
                if (++kp != t.k_blocks)
                    continue;
                kp = 0;
                if (!t.rem)
                    continue;
                int got = 0;
                if (lane == 0)
                    got = mbar_wait_bounded(smem_u32(&bars.tail[r.stage]), (parity >> r.stage) & 1u, abort_flag,
                                            args.wait_limit_ns)
                              ? 1
                              : 0;
                if (!__shfl_sync(kFull, got, 0)) {
                    ok = false;
                    break;
                }
                parity ^= 1u << r.stage;
                uint4 *const s = reinterpret_cast<uint4 *>(st.smem + r.stage * kStageBytes);
                const int n = ((t.rem + kUmmaK - 1) / kUmmaK * kUmmaK - t.rem) * 8;   // 16-byte words of a block to zero
                for (int i = lane; i < 4 * n; i += 32) {
                    const int block = i / n;
                    s[block * (kAtom / 16) + t.rem * 8 + (i - block * n)] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_release_cluster(map_to_cta(smem_u32(&bars.full[r.stage]), 0));
            }
        }
    } else if (warp >= 4) {
        const int q = warp - 4;
        float *const scratch = reinterpret_cast<float *>(st.smem + kStages * kStageBytes) + q * 32 * 36;
        int local = 0;
        for (int u = st.cluster; u < units; u += st.clusters, ++local) {
            const ProductUnit t = product_unit(u, args, s_off, s_tp);
            const ProductJob &j = args.job[t.job];
            const int buf = local & 1;
            int ok = 0;
            if (lane == 0)
                ok = mbar_wait_bounded(smem_u32(&bars.tfull[buf]), (local >> 1) & 1, abort_flag, args.wait_limit_ns) ? 1 : 0;
            if (!__shfl_sync(kFull, ok, 0))
                break;
            tc_fence_after();
            const uint32_t t_row = st.tmem + buf * 256 + (static_cast<uint32_t>(q * 32) << 16);
            const size_t base = (j.by_rows ? 0 : static_cast<size_t>(t.e) * j.expert_stride) + static_cast<size_t>(t.m0) * j.ld;
            if (t.k_blocks || !j.accumulate)
                store_rows(t_row, scratch, j, base, 128 * static_cast<int>(st.rank) + q * 32, t.rows, t.n0, t.k_blocks == 0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(map_to_cta(smem_u32(&bars.tempty[buf]), 0));
        }
    }
    pair_end(st, s_abort, args.err);
}

// ------------------------------------------------------------------ host side

// Launch a CTA-pair kernel with at most `units` pairs. The attribute and the
// occupancy are looked up once per host thread, device and kernel.
template <typename Args>
cudaError_t launch_pair(void (*kern)(Args), const Args &args, long long units, int num_sms, cudaStream_t stream)
{
    static thread_local int done_for_device = -1;
    static thread_local int max_clusters = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kDynSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (done_for_device != dev) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynSmem)) != cudaSuccess)
            return e;
        cfg.gridDim = dim3(2 * (num_sms / 2));
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess)
            return e;
        max_clusters = n > 0 ? n : 1;
        done_for_device = dev;
    }
    const long long clusters = units < 1 ? 1 : (units < max_clusters ? units : max_clusters);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters));
    return cudaLaunchKernelEx(&cfg, kern, args);
}

long long tiles_of(long long n) { return (n + 255) / 256; }

}  // namespace

long long product_units(const ProductJob &j, int E, int cap)
{
    return j.by_rows ? (tiles_of(cap) + E) * tiles_of(j.N) : E * tiles_of(j.M) * tiles_of(j.N);
}

cudaError_t launch_products(const ProductJob *jobs, int n, const int32_t *offsets, int E, int cap, int32_t *err,
                            int num_sms, cudaStream_t stream)
{
    ProductArgs a = {};
    long long units = 0;
    for (int i = 0; i < n; ++i) {
        const ProductJob &j = jobs[i];
        a.job[i] = j;
        if (!make_tile_map(&a.map[2 * i], j.a, static_cast<uint64_t>(j.a_rows), static_cast<uint64_t>(j.a_cols),
                           j.by_rows ? 128 : 64) ||
            !make_tile_map(&a.map[2 * i + 1], j.b, static_cast<uint64_t>(j.b_rows), static_cast<uint64_t>(j.b_cols), 64))
            return cudaErrorInvalidValue;
        units += product_units(j, E, cap);
    }
    a.jobs = n;
    a.offsets = offsets;
    a.E = E;
    a.cap = cap;
    a.err = err;
    a.wait_limit_ns = kWaitLimitNs;
    return launch_pair(products_kernel, a, units, num_sms, stream);
}

cudaError_t launch_act_grad(const void *x, const void *dy, const void *W13, const void *W2, const int32_t *offsets,
                            int E, int cap, int H, int I, void *act, void *dgu, int32_t *err, int num_sms,
                            cudaStream_t stream)
{
    ActArgs a = {};
    const uint64_t rows = cap, h = H, i = I, e = E;
    if (!make_tile_map(&a.x, x, rows, h, 128) || !make_tile_map(&a.dy, dy, rows, h, 128) ||
        !make_tile_map(&a.w13, W13, e * 2 * i, h, 128) || !make_tile_map(&a.w2, W2, e * h, i, 64))
        return cudaErrorInvalidValue;
    a.offsets = offsets;
    a.err = err;
    a.act = static_cast<__nv_bfloat16 *>(act);
    a.dgu = static_cast<__nv_bfloat16 *>(dgu);
    a.wait_limit_ns = kWaitLimitNs;
    a.E = E;
    a.cap = cap;
    a.H = H;
    a.I = I;
    return launch_pair(act_grad_kernel, a, (tiles_of(cap) + E) * ((I + 127) / 128), num_sms, stream);
}

}  // namespace moe
