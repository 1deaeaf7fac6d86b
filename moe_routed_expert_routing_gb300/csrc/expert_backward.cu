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
// stored. As K rows (weight gradients) they must not count, whatever they hold:
// another expert's rows or, past the valid ones, anything. Of an expert's last K
// block only its own rows are loaded, 16 at a time (the K of one MMA) and the
// last of them one by one (tile::gather4), filled up to 16 with a row of zeros
// that the workspace keeps behind a, [dg du] and the router's gradient, against
// the expert's own last row in the other operand. (Zeroing the rows in shared
// memory instead, by a warp between the copy and the MMAs, cost about 1 us for
// every tile of 256 x 256, in a loop that waits for its copies: dW13 at T=8192,
// E=128, H=4096, I=1536 1.69 ms, so 1.27.)
#include <cuda_bf16.h>

#include "moe_internal.h"
#include "ptx.cuh"
#include "tiles.cuh"

namespace moe {

namespace {

constexpr int kBK = 64;                      // K elements of a stage
constexpr int kUmmaK = 16;
constexpr int kTileRows = 256;               // rows of a CTA pair's tile
constexpr int kRowBox = 32;                  // rows of a box of a partial tile
constexpr int kHalf = 128 * 128;             // bytes of one operand's half tile: 128 x 64 bf16
constexpr int kStageBytes = 2 * kHalf;        // A, then B
constexpr int kAtom = 64 * 128;              // bytes of an MN-major block: 64 K rows x 64 columns
constexpr int kBox = 32 * 128;               // bytes of an output box: 32 rows x 128 bytes

// A kernel's pipeline stages and epilogue warps: four, one for each quarter of
// the TMEM lanes, or eight, each with half the columns.
template <int kStages_, int kWarps_, bool kBoxes, bool kSplit_ = false>
struct Config {
    static constexpr int kStages = kStages_, kWarps = kWarps_;
    static constexpr bool kSplit = kSplit_;      // tiles of up to 128 rows in halves
    static constexpr int kThreads = 128 + 32 * kWarps;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + (kBoxes ? kWarps * kBox : 0);
};
using ActConfig = Config<6, 8, false>;
// At most 128 rows an expert on average: a tile of up to 128 rows is split between the
// CTAs, in one box of 32 or 64 rows each. Its rows then take at most half of a stage's A,
// and two K blocks of da go into one stage: each brings 8 KB of W2 only, too little on
// its way at six stages. act_grad_kernel, E=50, 1000 tokens of 6 experts, H=2880, I=1472
// 261 -> 250 us; E=32, 32 rows an expert, H=2048, I=1024 107.5 -> 98.5. With whole tiles beside
// them such halves cost (E=128, 256 rows an expert, H=4096, I=1536, both kernels 3.40 and
// 3.51 ms). (Tiles of 32 rows up to 24 rows an expert, with more stages of weights on their way,
// gained 1 to 3% where every expert has as many rows, but an expert of many rows then fetches its
// weights for every 32 of them, and the host does not know: E=128, H=2048, I=1024, 16 rows on average 702
// and 710 us, with shares of 1 / rank^1.2 734 and 691; E=64, H=4096, I=1536, 24 rows 1067 and
// 1078, 1200 and 1107.)
using SplitConfig = Config<6, 8, false, true>;
constexpr int kSplitRows = 128;
using DeepConfig = Config<6, 4, true>;       // products: more copies in flight
// Products with eight epilogue warps, us beside those with DeepConfig:
//  * few rows an expert, where the weight gradients' tiles have one or two K blocks and wait for
//    their epilogue: E=32, H=2048, I=1024 at 16, 32 and 64 rows an expert 201 / 219, 207 / 221 and
//    212 / 225; E=50, 120 rows, H=2880, I=1472 679 / 684; E=128, H=4096, I=1536 at 128 rows 2521 /
//    2513, 180 rows 2820 / 2715, 512 rows 5710 / 5600;
//  * small problems, where each unit's way from its first copy to its last store counts: H=1024, I=512,
//    160 rows an expert with 1.5, 4.4, 5.9 and 8.8 units a pair 26.6 / 27.3, 36.3 / 37.6, 43.9 / 44.4 and
//    63.6 / 63.9; the router's E=384, H=7168 at T=257, 500, 1000 and 2000 20.7 / 21.7, 22.1 / 22.9, 28.7 / 28.5
//    and 46.2 / 44.9. More rows an expert give some of it back: 256 rows with 1.5, 2.9, 5.9 and 8.8 units 25.9 /
//    26.8, 33.0 / 32.9, 57.8 / 56.2 and 70.5 / 68.6, 512 rows with 0.8, 1.7 and 5.1 25.7 / 25.9, 29.5 / 29.0
//    and 58.7 / 56.7;
//  * few K blocks of a tile of rows, the router's dx (twice E / 64): T=8192, H=4096 with E=64, 128 and
//    256 42.5 / 44.8, 48.0 / 49.0 and 66.4 / 64.8.
using WideConfig = Config<5, 8, true>;
constexpr int kWideRows = 128;               // up to so many rows an expert on average
constexpr int kWideUnits = 6;                // or units a CTA pair
constexpr int kWideBlocks = 4;               // or K blocks of a tile of rows
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

// tma_gather4 completing an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap *map, uint32_t cluster_bar, int32_t c0,
                                                 const int (&rows)[4], uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
                 ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(rows[0]), "r"(rows[1]), "r"(rows[2]), "r"(rows[3]),
                 "r"(cluster_bar), "l"(policy)
                 : "memory");
}

__device__ __forceinline__ void fence_proxy_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 32 bytes of one row, 32-byte aligned: whole sectors.
__device__ __forceinline__ void store32(void *p, const uint32_t *v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// A box out of shared memory, stored or (fp32) added; one bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int32_t c0, int32_t c1, bool add)
{
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(c0), "r"(c1), "r"(src)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(c0), "r"(c1), "r"(src)
                     : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// until this thread's bulk groups have read shared memory
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Rows of a tile in the first CTA of its pair.
template <bool kSplit>
__device__ __forceinline__ int first_rows(int rows)
{
    return kSplit && rows <= 128 ? (rows <= 64 ? 32 : 64) : 128;
}

// The rows of a tile that this CTA's half of A needs, `n` of 128, as whole 32-row
// boxes, or one box where all are there. MMA rows past them keep whatever the
// stage held before: they are never stored.
__device__ __forceinline__ int boxed_rows(int n) { return n <= 0 ? 0 : (n >= 128 ? 128 : (n + kRowBox - 1) / kRowBox * kRowBox); }

__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, const CUtensorMap *map32, uint32_t full,
                                          int col, int row, int boxed, uint64_t policy)
{
    if (boxed == 128)
        tma_load_2d_pair(dst, map, full, col, row, policy);
    else
        for (int i = 0; i < boxed; i += kRowBox)
            tma_load_2d_pair(dst + i * 128, map32, full, col, row + i, policy);
}

// What every thread of a CTA pair's kernel starts from.
struct PairState {
    uint8_t *smem;          // stages, then the output boxes; 1024-byte aligned
    uint32_t tmem;
    uint32_t rank;
    int cluster, clusters;
};

template <int kStages>
struct PairBars {
    uint64_t full[kStages];    // used in CTA 0: one arrival and the bytes of each CTA
    uint64_t empty[kStages];
    uint64_t tfull[2];
    uint64_t tempty[2];        // used in CTA 0
    uint64_t drain;            // used in CTA 0
    uint64_t ufull[2], uempty[2];   // batches of units
};

// Barriers and TMEM. The offsets are read and the units decoded by one warp
// (load_offsets), while the others wait for the first units. Reads no global memory.
template <class C>
__device__ __forceinline__ PairState pair_begin(uint8_t *smem_raw, PairBars<C::kStages> &bars, uint32_t &s_tmem, int &s_abort)
{
    PairState st;
    st.smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    st.rank = cluster_ctarank();
    st.cluster = blockIdx.x >> 1;
    st.clusters = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 2);
            mbar_init(smem_u32(&bars.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bars.tfull[b]), 1);
            mbar_init(smem_u32(&bars.tempty[b]), 2 * C::kWarps);   // both CTAs' epilogue warps
            mbar_init(smem_u32(&bars.ufull[b]), 1);
            mbar_init(smem_u32(&bars.uempty[b]), C::kWarps + (st.rank ? 1 : 2));   // loads, MMAs (CTA 0), epilogue
        }
        mbar_init(smem_u32(&bars.drain), 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if ((threadIdx.x >> 5) == 2) {
        tmem_alloc_pair(smem_u32(&s_tmem), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers initialised before any remote arrive
    tc_fence_after();
    st.tmem = s_tmem;
    return st;
}

// A warp: the experts' offsets, clamped to the batch, and their row tiles.
__device__ __forceinline__ void load_offsets(const int32_t *offsets, int E, int cap, int *s_off, int *s_tp)
{
    const int lane = threadIdx.x & 31;
    for (int i = lane; i <= E; i += 32) {
        const int o = offsets[i];
        s_off[i] = o < 0 ? 0 : (o > cap ? cap : o);
    }
    __syncwarp();
    build_tile_prefix(s_off, s_tp, E, kTileRows, lane);
    __syncwarp();
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

// The MMAs of `steps` times 16 K elements of one stage. The majors are known when
// it is compiled: one thread issues a pair's MMAs, in 256 to 512 cycles a stage,
// and a branch between the steps (the router's second part beside the plain
// step) cost the products a third of their rate: dx at E=16, T=8192, H=4096, I=1536
// 1.29 ms and 0.93.
template <bool kAMn, bool kBMn>
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t a_addr, uint32_t idesc, bool first, int steps)
{
    constexpr uint32_t kA = kAMn ? 2048 >> 4 : 32 >> 4, kB = kBMn ? 2048 >> 4 : 32 >> 4;
    const uint32_t b_addr = a_addr + kHalf;
    const uint64_t a0 = kAMn ? smem_desc_mnmajor_sw128(a_addr) : smem_desc_kmajor_sw128(a_addr);
    const uint64_t b0 = kBMn ? smem_desc_mnmajor_sw128(b_addr) : smem_desc_kmajor_sw128(b_addr);
    if (steps == kBK / kUmmaK) {
        umma_bf16_pair(d, a0, b0, idesc, first ? 0u : 1u);
#pragma unroll
        for (int kk = 1; kk < kBK / kUmmaK; ++kk)
            umma_bf16_pair(d, a0 + kk * kA, b0 + kk * kB, idesc, 1u);
    } else {
        for (int kk = 0; kk < steps; ++kk)
            umma_bf16_pair(d, a0 + kk * kA, b0 + kk * kB, idesc, (first && kk == 0) ? 0u : 1u);
    }
}

template <int kStages>
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

// ------------------------------------------------------------------ units

// A unit of work, decoded. A warp of its own decodes 32 units at a time, one a
// lane, into one of two batches in shared memory, and every role reads them
// from there: decoding takes some 2 us of divisions and searches, which each
// role spent between two units before (with it and TMA stores: T=8192,
// E=128, H=4096, I=1536 6.25 -> 5.63 ms; E=50, T=1000 1.00 -> 0.73 ms).
struct __align__(16) UnitDesc {
    int job;             // products: which; -1: no more units
    int e;
    int m0, n0;          // first row and column of the output tile
    int rows;            // output rows of the tile that exist
    int total;           // K blocks
    int period;          // after how many of them B begins again
    int rem;             // rows of the last K block when that is not whole, else 0
    int k_row0;          // first K row, where K runs along the batch
    int pad[3];
};

constexpr int kBatch = 32;

struct UnitReader {
    const UnitDesc *units;
    uint64_t *full, *empty;
    int i;
    __device__ __forceinline__ UnitReader(const UnitDesc *u, uint64_t *f, uint64_t *e) : units(u), full(f), empty(e), i(0) {}
    // One thread: the next unit, or null at the end or on give-up.
    __device__ __forceinline__ const UnitDesc *next(volatile int *abort, uint64_t limit_ns)
    {
        const int b = (i / kBatch) & 1;
        if (i % kBatch == 0) {
            if (i)
                mbar_arrive(smem_u32(&empty[b ^ 1]));    // the batch before has been used
            if (!mbar_wait_bounded(smem_u32(&full[b]), (i / (2 * kBatch)) & 1, abort, limit_ns))
                return nullptr;
        }
        const UnitDesc *u = units + b * kBatch + i % kBatch;
        ++i;
        return u->job < 0 ? nullptr : u;
    }
    // A warp: lane 0 waits.
    __device__ __forceinline__ const UnitDesc *next_warp(int lane, volatile int *abort, uint64_t limit_ns)
    {
        const int b = (i / kBatch) & 1;
        if (i % kBatch == 0) {
            int ok = 0;
            __syncwarp();
            if (lane == 0) {
                if (i)
                    mbar_arrive(smem_u32(&empty[b ^ 1]));
                ok = mbar_wait_bounded(smem_u32(&full[b]), (i / (2 * kBatch)) & 1, abort, limit_ns) ? 1 : 0;
            }
            if (!__shfl_sync(kFull, ok, 0))
                return nullptr;
            __syncwarp();
        }
        const UnitDesc *u = units + b * kBatch + i % kBatch;
        ++i;
        return u->job < 0 ? nullptr : u;
    }
};

// The decoding warp: units st.cluster, st.cluster + st.clusters, ... below `units`.
template <int kStages, typename Decode>
__device__ __forceinline__ void publish_units(const PairState &st, PairBars<kStages> &bars, UnitDesc *s_units, int units,
                                              volatile int *abort, uint64_t limit_ns, Decode decode)
{
    const int lane = threadIdx.x & 31;
    long long u = st.cluster + static_cast<long long>(lane) * st.clusters;
    for (int batch = 0;; ++batch, u += static_cast<long long>(kBatch) * st.clusters) {
        const int b = batch & 1;
        int ok = 0;
        if (batch == 2)
            pdl_wait();    // the first two wait for nobody: no limit runs while the kernel ahead does
        if (lane == 0)
            ok = mbar_wait_bounded(smem_u32(&bars.uempty[b]), ((batch >> 1) & 1) ^ 1u, abort, limit_ns) ? 1 : 0;
        if (!__shfl_sync(kFull, ok, 0))
            return;
        UnitDesc d = {};
        d.job = -1;
        if (u < units)
            decode(static_cast<int>(u), d);
        s_units[b * kBatch + lane] = d;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&bars.ufull[b]));
        if (__any_sync(kFull, u >= units))
            return;
    }
}

// 32 rows x 128 bytes of an epilogue warp's box at `box` (128-byte swizzle),
// rows [first, first + 32) of a tile with `rows` of them, to element (c0, r0 +
// first) of `map`; boxes that hold rows past the tile go row by row. (Only the rows of
// a batch end inside a box, and only weight gradients, whose tiles are whole
// boxes, are added.)
__device__ __forceinline__ void store_box(uint8_t *box, const CUtensorMap *map, int c0, int r0, int first, int rows,
                                          void *out, long long ld, int esize, bool add)
{
    const int lane = threadIdx.x & 31;
    if (first >= rows)
        return;
    if (first + 32 <= rows) {
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, smem_u32(box), c0, r0 + first, add);
            bulk_commit();
        }
        return;
    }
    __syncwarp();
#pragma unroll
    for (int it = 0; it < 8; ++it) {
        const int rr = 4 * it + (lane >> 3), ch = lane & 7;
        if (first + rr < rows)
            *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(out) +
                                       ((static_cast<long long>(r0) + first + rr) * ld + c0) * esize + ch * 16) =
                *reinterpret_cast<const uint4 *>(box + rr * 128 + ((ch ^ (rr & 7)) << 4));
    }
    __syncwarp();
}

// ------------------------------------------------------------------ a and [dg du]

struct ActArgs {
    CUtensorMap x, dy;       // [cap, H], boxes of 64 x 128 rows
    CUtensorMap x32, dy32;   // the same in boxes of 64 x 32 rows
    CUtensorMap w13;         // [E * 2I, H], boxes of 64 x 128 rows
    CUtensorMap w2;          // [E * H, I], boxes of 64 x 64 rows
    CUtensorMap x64, dy64, w2_two;   // split tiles: boxes of 64 x 64 rows, of 64 x 128 rows
    const int32_t *offsets;
    int32_t *err;
    __nv_bfloat16 *act;      // [cap + 1, I]: the last row is zeros
    __nv_bfloat16 *dgu;      // [cap + 1, 2I]
    uint64_t wait_limit_ns;
    int E, cap, H, I;
};

// Column tile, then row tile: the row tiles that share one weight tile go to
// neighbouring pairs. (A last tile of at most 128 rows turned round, weights on
// the MMAs' M side and its rows on N, saves MMAs on padding, but with partial
// tiles that load only their rows it does not pay: 256 rows an expert, E=128, H=4096,
// I=1536 3.48 ms with it and 3.35 without, 120 rows 702 us and 690; only very few long
// ones gain, 10 rows of each of 5 experts, H=3904, I=960 92 us and 100.)
__device__ __forceinline__ void act_unit(int u, UnitDesc &d, const int *s_off, const int *s_tp, int E, int NT)
{
    const int e = find_expert(s_tp, E, u, NT);
    const int local = u - s_tp[e] * NT;
    const int tiles = s_tp[e + 1] - s_tp[e];
    const int nt = local / tiles;
    d.job = 0;
    d.e = e;
    d.m0 = s_off[e] + (local - nt * tiles) * kTileRows;
    d.rows = min(s_off[e + 1] - d.m0, kTileRows);
    d.n0 = nt * 128;
}

// One element's gradients from its gate, up and da values. The fast exponential is off
// by up to (2 + 1.16 |g|) 2^-23, 1e-5 at |g| = 80, the quotient by 2^-22: far below the
// rounding to bf16 behind them, 2^-8. Below g = -87 s is 0 where it is 1e-38 and less.
__device__ __forceinline__ void swiglu_grad(float g, float u, float d, float &a, float &dg, float &du)
{
    const float s = __fdividef(1.0f, 1.0f + __expf(-g));
    const float silu = g * s;
    a = silu * u;
    du = d * silu;
    dg = d * u * (s * (1.0f + g * (1.0f - s)));
}

// TMEM columns: da of even and odd units in 0..127 and 128..255, gate and up
// in 256..383 and 384..511. A unit's da comes first, so that it can be
// multiplied while the unit before is still being read out: a third of the
// unit's MMAs, which hides that unit's epilogue.
template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) act_grad_kernel(const __grid_constant__ ActArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) PairBars<C::kStages> bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_off[kMaxExperts + 1];
    __shared__ int s_tp[kMaxExperts + 1];
    __shared__ UnitDesc s_units[2 * kBatch];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NT = (args.I + 127) / 128;
    const PairState st = pair_begin<C>(smem_raw, bars, s_tmem, s_abort);
    pdl_wait();
    volatile int *abort_flag = &s_abort;
    const int k_blocks = args.H / kBK;
    pdl_trigger();    // the products' CTAs need this kernel's shared memory: each starts as one here ends
    if (blockIdx.x == 0 && warp == 3) {
        // the rows of zeros behind a and [dg du]
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int i = lane; i < args.I / 8; i += 32)
            reinterpret_cast<uint4 *>(args.act + static_cast<size_t>(args.cap) * args.I)[i] = zero;
        for (int i = lane; i < args.I / 4; i += 32)
            reinterpret_cast<uint4 *>(args.dgu + static_cast<size_t>(args.cap) * 2 * args.I)[i] = zero;
    }
    const int rank = static_cast<int>(st.rank);

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_w = l2_policy_evict_normal();
            const uint64_t pol_a = l2_policy_evict_last();
            Ring<C::kStages> r;
            UnitReader units(s_units, bars.ufull, bars.uempty);
            bool ok = true;
            while (const UnitDesc *t = ok ? units.next(abort_flag, args.wait_limit_ns) : nullptr) {
                const int n0 = t->n0;
                const int split = first_rows<C::kSplit>(t->rows);
                const int a_row = t->m0 + split * rank;
                const int boxed = split == 64 ? 64 : boxed_rows(rank ? t->rows - split : min(t->rows, split));
                const int per = split < 128 ? 2 : 1;               // K blocks of da in a stage
                const int w2_row = t->e * args.H;
                const int w13_row = t->e * 2 * args.I + n0 + (rank ? args.I : 0);
                for (int kb = 0; kb < 2 * k_blocks; kb += kb < k_blocks ? min(per, k_blocks - kb) : 1, r.next()) {
                    if (!mbar_wait_bounded(smem_u32(&bars.empty[r.stage]), r.phase ^ 1u, abort_flag,
                                           args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = map_to_cta(smem_u32(&bars.full[r.stage]), 0);
                    const uint32_t a_dst = smem_u32(st.smem + r.stage * kStageBytes);
                    const uint32_t b_dst = a_dst + kHalf;
                    if (kb < k_blocks) {
                        const int kc = kb * kBK;
                        if (C::kSplit && split < 128) {
                            const int n = min(per, k_blocks - kb);
                            const CUtensorMap *const part = split == 64 ? &args.dy64 : &args.dy32;
                            mbar_arrive_expect_tx_cluster(full, n * (boxed * 128 + kAtom));
                            tma_load_2d_pair(b_dst, n == 2 ? &args.w2_two : &args.w2, full, n0 + 64 * rank, w2_row + kc, pol_w);
                            for (int i = 0; boxed && i < n; ++i)
                                tma_load_2d_pair(a_dst + i * kAtom, part, full, kc + i * kBK, a_row, pol_a);
                        } else {
                            mbar_arrive_expect_tx_cluster(full, boxed * 128 + kAtom);
                            load_rows(a_dst, &args.dy, &args.dy32, full, kc, a_row, boxed, pol_a);
                            tma_load_2d_pair(b_dst, &args.w2, full, n0 + 64 * rank, w2_row + kc, pol_w);
                        }
                    } else {
                        const int kc = (kb - k_blocks) * kBK;
                        mbar_arrive_expect_tx_cluster(full, boxed * 128 + kHalf);
                        if (C::kSplit && split == 64)
                            tma_load_2d_pair(a_dst, &args.x64, full, kc, a_row, pol_a);
                        else
                            load_rows(a_dst, &args.x, &args.x32, full, kc, a_row, boxed, pol_a);
                        tma_load_2d_pair(b_dst, &args.w13, full, kc, w13_row, pol_w);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && st.rank == 0) {
            Ring<C::kStages> r;
            UnitReader units(s_units, bars.ufull, bars.uempty);
            bool ok = true;
            int local = 0;
            while (const UnitDesc *t = ok ? units.next(abort_flag, args.wait_limit_ns) : nullptr) {
                const int per = first_rows<C::kSplit>(t->rows) < 128 ? 2 : 1;
                // da, then gate and up, once those of the unit before have been read (and with them the da before that)
                constexpr uint32_t kIdescDa = idesc_bf16_f32(256, 128) | kMajorB, kIdescGu = idesc_bf16_f32(256, 256);
                const uint32_t d_da = st.tmem + 128 * (local & 1), d_gu = st.tmem + 256;
                for (int kb = 0; kb < k_blocks; kb += per, r.next()) {
                    if (!mbar_wait_bounded(smem_u32(&bars.full[r.stage]), r.phase, abort_flag, args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(st.smem + r.stage * kStageBytes);
                    mma_stage<false, true>(d_da, a_addr, kIdescDa, kb == 0, 4);
                    if (per == 2 && kb + 1 < k_blocks)      // A's second half tile is 64 rows behind, as B's is
                        mma_stage<false, true>(d_da, a_addr + kAtom, kIdescDa, false, 4);
                    umma_commit_pair(smem_u32(&bars.empty[r.stage]), 0x3);
                }
                if (!ok || !mbar_wait_bounded(smem_u32(&bars.tempty[0]), (local & 1) ^ 1u, abort_flag,
                                              args.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                for (int kb = 0; kb < k_blocks; ++kb, r.next()) {
                    if (!mbar_wait_bounded(smem_u32(&bars.full[r.stage]), r.phase, abort_flag, args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mma_stage<false, false>(d_gu, smem_u32(st.smem + r.stage * kStageBytes), kIdescGu, kb == 0, 4);
                    umma_commit_pair(smem_u32(&bars.empty[r.stage]), 0x3);
                }
                if (ok)
                    umma_commit_pair(smem_u32(&bars.tfull[0]), 0x3);
                ++local;
            }
            umma_commit_pair(smem_u32(&bars.drain), 0x1);
            mbar_drain(smem_u32(&bars.drain), 0, args.wait_limit_ns);
        }
        __syncwarp();
    } else if (warp == 2) {
        load_offsets(args.offsets, args.E, args.cap, s_off, s_tp);
        publish_units(st, bars, s_units, s_tp[args.E] * NT, abort_flag, args.wait_limit_ns, [&](int u, UnitDesc &d) {
            act_unit(u, d, s_off, s_tp, args.E, NT);
        });
    } else if (warp >= 4) {
        const int q = warp & 3, half = (warp - 4) >> 2;
        UnitReader units(s_units, bars.ufull, bars.uempty);
        int local = 0;
        for (; const UnitDesc *tp = units.next_warp(lane, abort_flag, args.wait_limit_ns); ++local) {
            const UnitDesc t = *tp;
            int ok = 0;
            if (lane == 0)
                ok = mbar_wait_bounded(smem_u32(&bars.tfull[0]), local & 1, abort_flag, args.wait_limit_ns) ? 1 : 0;
            if (!__shfl_sync(kFull, ok, 0))
                break;
            tc_fence_after();
            const uint32_t lanes = st.tmem + (static_cast<uint32_t>(q * 32) << 16);
            const uint32_t t_da = lanes + 128 * (local & 1), t_gu = lanes + 256;
            const int split = first_rows<C::kSplit>(t.rows);
            const int r = split * rank + q * 32 + lane;
            const bool valid = r < (rank ? t.rows : min(t.rows, split));
            const int cols = min(args.I - t.n0, 128);     // a multiple of 64
            __nv_bfloat16 *const act = args.act + static_cast<size_t>(t.m0 + r) * args.I + t.n0;
            __nv_bfloat16 *const dgu = args.dgu + static_cast<size_t>(t.m0 + r) * 2 * args.I + t.n0;
#pragma unroll 1
            for (int c = 64 * half; c < cols && c < 64 * half + 64; c += 16) {
                uint32_t vg[16], vu[16], vd[16];
                tmem_ld_32x32b_x16(t_gu + c, vg);
                tmem_ld_32x32b_x16(t_gu + 128 + c, vu);
                tmem_ld_32x32b_x16(t_da + c, vd);
                tmem_wait_ld();
                uint32_t o[3][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float a[2], g[2], w[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        swiglu_grad(__uint_as_float(vg[2 * i + j]), __uint_as_float(vu[2 * i + j]),
                                    __uint_as_float(vd[2 * i + j]), a[j], g[j], w[j]);
                    o[0][i] = pack_bf16x2(a[0], a[1]);
                    o[1][i] = pack_bf16x2(g[0], g[1]);
                    o[2][i] = pack_bf16x2(w[0], w[1]);
                }
                if (valid) {   // the workspace is 256-byte aligned, its rows whole 128-byte lines
                    store32(act + c, o[0]);
                    store32(dgu + c, o[1]);
                    store32(dgu + args.I + c, o[2]);
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

struct ProductArgs {
    ProductJob job[3];
    CUtensorMap a[3], b[3], out[3];
    CUtensorMap a32[3];             // rows kind: A in boxes of 32 rows
    CUtensorMap a16[3], b16[3];     // weights kind: both in boxes of 16 rows
    CUtensorMap a1[3], b1[3];       // and of one row, for gathers
    const int32_t *offsets;
    int32_t *err;
    uint64_t wait_limit_ns;
    int jobs, E, cap;
    const int32_t *num_rows;        // segments: as many rows as there are (null: cap)
    int segment_rows;               // 0: ranges by `offsets`; else E segments of so many rows
};

__device__ __forceinline__ int job_units(const ProductJob &j, const int *s_tp, int E)
{
    const int tile_n = j.rows_on_n ? 128 : 256, NT = (j.N + tile_n - 1) / tile_n;
    return j.by_rows ? s_tp[E] * NT : E * ((j.M + 255) / 256) * NT;
}

__device__ __forceinline__ void product_unit(int u, UnitDesc &d, const ProductArgs &args, const int *s_off,
                                             const int *s_tp)
{
    int job = 0;
    for (; job + 1 < args.jobs; ++job) {
        const int n = job_units(args.job[job], s_tp, args.E);
        if (u < n)
            break;
        u -= n;
    }
    const ProductJob &j = args.job[job];
    const int tile_n = j.rows_on_n ? 128 : 256, NT = (j.N + tile_n - 1) / tile_n;
    d.job = job;
    if (j.by_rows) {
        const int rt = u / NT;
        d.n0 = (u - rt * NT) * 256;
        d.e = find_expert(s_tp, args.E, rt, 1);
        d.m0 = s_off[d.e] + (rt - s_tp[d.e]) * kTileRows;
        d.rows = min(s_off[d.e + 1] - d.m0, kTileRows);
        d.total = j.k_blocks;
        d.period = j.wrap;
    } else {
        const int MT = (j.M + 255) / 256;
        d.e = u / (MT * NT);
        u -= d.e * MT * NT;
        const int mt = u / NT;
        d.m0 = mt * 256;
        d.n0 = (u - mt * NT) * tile_n;
        d.rows = j.rows_on_n ? min(j.N - d.n0, 128) : min(j.M - d.m0, 256);
        const int k = max(s_off[d.e + 1] - s_off[d.e], 0);
        d.period = (k + kBK - 1) / kBK;
        d.total = d.period;
        d.rem = k % kBK;
        d.k_row0 = s_off[d.e];
    }
}

// Rows first .. first + 31 of a tile, columns c_begin .. c_end - 1, out of TMEM
// (or zeros) to memory, one box of 128-byte rows at a time.
__device__ __forceinline__ void store_tile(uint32_t t_row, uint8_t *box, const ProductJob &j,
                                           const CUtensorMap *map, int r0, int first, int rows, int n0, int c_begin,
                                           int c_end, bool zero)
{
    const int lane = threadIdx.x & 31;
    const int cols = min(j.N - n0, c_end);     // a multiple of 64
    const int step = j.out_f32 ? 32 : 64;
#pragma unroll 1
    for (int c = c_begin; c < cols; c += step) {
        uint32_t d[32];
        if (zero) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                d[i] = 0u;
        } else if (j.out_f32) {
            tmem_ld_32x32b_x32(t_row + c, d);
            tmem_wait_ld();
        } else {
            uint32_t v[64];
            tmem_ld_32x32b_x32(t_row + c, *reinterpret_cast<uint32_t(*)[32]>(v));
            tmem_ld_32x32b_x32(t_row + c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
                d[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        }
        if (lane == 0)
            bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(box + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_uint4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
        store_box(box, map, n0 + c, r0, first, rows, j.out, j.N, j.out_f32 ? 4 : 2, j.accumulate != 0);
    }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) products_kernel(const __grid_constant__ ProductArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) PairBars<C::kStages> bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_off[kMaxExperts + 1];
    __shared__ int s_tp[kMaxExperts + 1];
    __shared__ UnitDesc s_units[2 * kBatch];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PairState st = pair_begin<C>(smem_raw, bars, s_tmem, s_abort);
    // The decoding warp need not wait, so that the first units are ready when the kernel ahead ends
    // (E=6, 1884 tokens of 3 experts, H=256, I=128 20.1 -> 18.4 us, E=32, 16 rows an expert,
    // H=2048, I=1024 200.1 -> 197.8; the router's, T=8192, E=128, H=4096 48.2 -> 46.1).
    if (warp != 2)
        pdl_wait();
    volatile int *abort_flag = &s_abort;
    const int rank = static_cast<int>(st.rank);

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = l2_policy_evict_normal();
            Ring<C::kStages> r;
            UnitReader units(s_units, bars.ufull, bars.uempty);
            bool ok = true;
            while (const UnitDesc *tp = ok ? units.next(abort_flag, args.wait_limit_ns) : nullptr) {
                const UnitDesc t = *tp;
                const ProductJob &j = args.job[t.job];
                const CUtensorMap *ma = &args.a[t.job], *mb = &args.b[t.job], *ma32 = &args.a32[t.job];
                const bool by_rows = j.by_rows != 0;
                const bool on_n = j.rows_on_n != 0;
                // B's two blocks of 64 columns in this CTA: neighbours, or the two parts of 64 columns
                const int b_col = t.n0 + (on_n ? 64 : 128) * rank, b_next = on_n ? j.part_cols : 64;
                const int a_row = t.m0 + 128 * rank;                      // rows kind
                const int b_row0 = t.e * j.b_expert_rows;
                const int boxed = boxed_rows(t.rows - 128 * rank);
                const int a_col = t.m0 + 128 * rank;                      // weights kind
                int kp = 0;
                for (int kb = 0; kb < t.total; ++kb, r.next()) {
                    if (!mbar_wait_bounded(smem_u32(&bars.empty[r.stage]), r.phase ^ 1u, abort_flag,
                                           args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = map_to_cta(smem_u32(&bars.full[r.stage]), 0);
                    const uint32_t a_dst = smem_u32(st.smem + r.stage * kStageBytes);
                    const uint32_t b_dst = a_dst + kHalf;
                    if (by_rows) {
                        const int b_row = b_row0 + kp * kBK;
                        mbar_arrive_expect_tx_cluster(full, kHalf + boxed * 128);
                        tma_load_2d_pair(b_dst, mb, full, b_col, b_row, pol);
                        tma_load_2d_pair(b_dst + kAtom, mb, full, b_col + 64, b_row, pol);
                        load_rows(a_dst, ma, ma32, full, kb * kBK, a_row, boxed, pol);
                    } else {
                        const int row = t.k_row0 + kp * kBK;
                        if (t.rem && kp + 1 == t.period) {
                            // the rows there are, 16 at a time; the last of them row by row, filled up to 16
                            // with the row of zeros in one operand, the expert's last row in the other
                            const int slabs = (t.rem + kUmmaK - 1) / kUmmaK, whole = t.rem / kUmmaK;
                            mbar_arrive_expect_tx_cluster(full, slabs * 4 * kUmmaK * 128);
                            for (int i = 0; i < whole; ++i) {
                                const uint32_t o = i * kUmmaK * 128;
                                const int r16 = row + i * kUmmaK;
                                tma_load_2d_pair(a_dst + o, &args.a16[t.job], full, a_col, r16, pol);
                                tma_load_2d_pair(a_dst + kAtom + o, &args.a16[t.job], full, a_col + 64, r16, pol);
                                tma_load_2d_pair(b_dst + o, &args.b16[t.job], full, b_col, r16, pol);
                                tma_load_2d_pair(b_dst + kAtom + o, &args.b16[t.job], full, b_col + b_next, r16, pol);
                            }
                            if (whole < slabs) {
                                const int last = row + t.rem - 1;
                                const int fill_a = j.zero_in_a ? args.cap : last, fill_b = j.zero_in_a ? last : args.cap;
#pragma unroll 1
                                for (int q = 0; q < kUmmaK / 4; ++q) {
                                    int ra[4], rb[4];
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const int r0 = row + whole * kUmmaK + 4 * q + i;
                                        ra[i] = r0 <= last ? r0 : fill_a;
                                        rb[i] = r0 <= last ? r0 : fill_b;
                                    }
                                    const uint32_t o = (whole * kUmmaK + 4 * q) * 128;
                                    tma_gather4_pair(a_dst + o, &args.a1[t.job], full, a_col, ra, pol);
                                    tma_gather4_pair(a_dst + kAtom + o, &args.a1[t.job], full, a_col + 64, ra, pol);
                                    tma_gather4_pair(b_dst + o, &args.b1[t.job], full, b_col, rb, pol);
                                    tma_gather4_pair(b_dst + kAtom + o, &args.b1[t.job], full, b_col + b_next, rb, pol);
                                }
                            }
                        } else {
                            mbar_arrive_expect_tx_cluster(full, kStageBytes);
                            tma_load_2d_pair(a_dst, ma, full, a_col, row, pol);
                            tma_load_2d_pair(a_dst + kAtom, ma, full, a_col + 64, row, pol);
                            tma_load_2d_pair(b_dst, mb, full, b_col, row, pol);
                            tma_load_2d_pair(b_dst + kAtom, mb, full, b_col + b_next, row, pol);
                        }
                    }
                    if (++kp == t.period)
                        kp = 0;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && st.rank == 0) {
            Ring<C::kStages> r;
            UnitReader units(s_units, bars.ufull, bars.uempty);
            bool ok = true;
            int local = 0;
            while (const UnitDesc *tp = ok ? units.next(abort_flag, args.wait_limit_ns) : nullptr) {
                const int total = tp->total, rem = tp->rem;
                const bool by_rows = args.job[tp->job].by_rows != 0, on_n = args.job[tp->job].rows_on_n != 0;
                const int buf = local & 1;
                if (!mbar_wait_bounded(smem_u32(&bars.tempty[buf]), ((local >> 1) & 1) ^ 1u, abort_flag,
                                       args.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = st.tmem + buf * 256;
                for (int kb = 0; kb < total; ++kb, r.next()) {
                    if (!mbar_wait_bounded(smem_u32(&bars.full[r.stage]), r.phase, abort_flag, args.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(st.smem + r.stage * kStageBytes);
                    const int steps = (rem && kb + 1 == total) ? (rem + kUmmaK - 1) / kUmmaK : kBK / kUmmaK;
                    if (by_rows) {
                        mma_stage<false, true>(d, a_addr, idesc_bf16_f32(256, 256) | kMajorB, kb == 0, kBK / kUmmaK);
                    } else if (!on_n) {
                        mma_stage<true, true>(d, a_addr, idesc_bf16_f32(256, 256) | kMajorA | kMajorB, kb == 0, steps);
                    } else {
                        // both parts of B
                        constexpr uint32_t kIdesc = idesc_bf16_f32(256, 128) | kMajorA | kMajorB;
                        const uint64_t a0 = smem_desc_mnmajor_sw128(a_addr), b0 = smem_desc_mnmajor_sw128(a_addr + kHalf);
                        for (int kk = 0; kk < steps; ++kk) {
                            umma_bf16_pair(d, a0 + kk * 128, b0 + kk * 128, kIdesc, (kb > 0 || kk > 0) ? 1u : 0u);
                            umma_bf16_pair(d, a0 + kk * 128, b0 + (kAtom >> 4) + kk * 128, kIdesc, 1u);
                        }
                    }
                    umma_commit_pair(smem_u32(&bars.empty[r.stage]), 0x3);
                }
                if (ok)
                    umma_commit_pair(smem_u32(&bars.tfull[buf]), 0x3);
                ++local;
            }
            umma_commit_pair(smem_u32(&bars.drain), 0x1);
            mbar_drain(smem_u32(&bars.drain), 0, args.wait_limit_ns);
        }
        __syncwarp();
    } else if (warp == 2) {
        if (args.segment_rows) {
            const int n = args.num_rows ? min(max(*args.num_rows, 0), args.cap) : args.cap;
            for (int i = lane; i <= args.E; i += 32)
                s_off[i] = static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(i) * args.segment_rows));
            __syncwarp();
            build_tile_prefix(s_off, s_tp, args.E, kTileRows, lane);
            __syncwarp();
        } else {
            load_offsets(args.offsets, args.E, args.cap, s_off, s_tp);
        }
        int units = 0;
        for (int j = 0; j < args.jobs; ++j)
            units += job_units(args.job[j], s_tp, args.E);
        publish_units(st, bars, s_units, units, abort_flag, args.wait_limit_ns, [&](int u, UnitDesc &d) {
            product_unit(u, d, args, s_off, s_tp);
        });
    } else if (warp >= 4) {
        const int q = warp & 3, half = (warp - 4) >> 2;
        constexpr int kHalves = C::kWarps / 4;
        uint8_t *const box = st.smem + C::kStages * kStageBytes + (warp - 4) * kBox;
        UnitReader units(s_units, bars.ufull, bars.uempty);
        int local = 0;
        for (; const UnitDesc *tp = units.next_warp(lane, abort_flag, args.wait_limit_ns); ++local) {
            const UnitDesc t = *tp;
            const ProductJob &j = args.job[t.job];
            const int buf = local & 1;
            int ok = 0;
            if (lane == 0)
                ok = mbar_wait_bounded(smem_u32(&bars.tfull[buf]), (local >> 1) & 1, abort_flag, args.wait_limit_ns) ? 1 : 0;
            if (!__shfl_sync(kFull, ok, 0))
                break;
            tc_fence_after();
            const uint32_t t_row = st.tmem + buf * 256 + (static_cast<uint32_t>(q * 32) << 16);
            if (!j.rows_on_n) {
                const int r0 = t.m0 + (j.by_rows ? 0 : t.e * j.M);
                if (t.total || !j.accumulate)
                    store_tile(t_row, box, j, &args.out[t.job], r0, 128 * rank + q * 32, t.rows, t.n0, half * 128,
                               kHalves == 1 ? 256 : half * 128 + 128, t.total == 0);
            } else {
                // lane = column (a row of the MMA's M side), TMEM columns = the unit's rows
                const int col = t.m0 + 128 * rank + q * 32 + lane, cols = j.M;
                const size_t row0 = static_cast<size_t>(t.e) * j.N + t.n0;
                const bool col_ok = col < cols;
#pragma unroll 1
                for (int c = 16 * half; c < t.rows; c += 16 * kHalves) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(t_row + c, v);
                    tmem_wait_ld();
                    if (t.total == 0)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] = 0u;
                    const int n = col_ok ? t.rows - c : 0;      // rows of these 16 to store
                    if (j.out_f32) {
                        float *p = static_cast<float *>(j.out) + (row0 + c) * cols + col;
#pragma unroll
                        for (int i = 0; i < 16; ++i, p += cols)
                            if (i < n)
                                *p = __uint_as_float(v[i]);
                    } else {
                        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(j.out) + (row0 + c) * cols + col;
#pragma unroll
                        for (int i = 0; i < 16; ++i, p += cols)
                            if (i < n)
                                *p = __float2bfloat16_rn(__uint_as_float(v[i]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(map_to_cta(smem_u32(&bars.tempty[buf]), 0));
        }
        if (lane == 0)
            bulk_wait_all();
        __syncwarp();
    }
    // The decoding warp may get here while the kernel ahead still runs, and one thread's trigger
    // counts for its CTA: no dependent may start before that kernel has completed.
    pdl_wait();
    pdl_trigger();
    pair_end(st, s_abort, args.err);
}

// ------------------------------------------------------------------ host side

// Launch a CTA-pair kernel with at most `units` pairs. The attribute and the
// occupancy are looked up once per host thread, device and kernel (each has a
// configuration type of its own).
template <class C, typename Args>
cudaError_t launch_pair(void (*kern)(Args), const Args &args, long long units, int num_sms, cudaStream_t stream)
{
    static thread_local int done_for_device = -1;
    static thread_local int max_clusters = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (done_for_device != dev) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) != cudaSuccess)
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
    return j.by_rows ? (tiles_of(cap) + E) * tiles_of(j.N)
                     : E * tiles_of(j.M) * (j.rows_on_n ? (j.N + 127LL) / 128 : tiles_of(j.N));
}

cudaError_t launch_products(const ProductJob *jobs, int n, const ProductRows &rows, int E, int cap, int32_t *err,
                            int num_sms, cudaStream_t stream)
{
    ProductArgs a = {};
    long long units = 0, live = 0;
    bool shallow = false;
    for (int i = 0; i < n; ++i) {
        const ProductJob &j = jobs[i];
        a.job[i] = j;
        const uint64_t a_rows = j.a_rows, a_cols = j.a_cols;
        const uint64_t out_rows = j.by_rows ? static_cast<uint64_t>(cap) : static_cast<uint64_t>(E) * j.M;
        const uint64_t b_rows = j.b_rows, b_cols = j.b_cols;
        if (!make_tile_map(&a.a[i], j.a, a_rows, a_cols, j.by_rows ? 128 : 64) ||
            (j.by_rows && !make_tile_map(&a.a32[i], j.a, a_rows, a_cols, kRowBox)) ||
            (!j.by_rows && (!make_tile_map(&a.a16[i], j.a, a_rows, a_cols, kUmmaK) ||
                            !make_tile_map(&a.b16[i], j.b, b_rows, b_cols, kUmmaK) ||
                            !make_tile_map(&a.a1[i], j.a, a_rows, a_cols, 1) ||
                            !make_tile_map(&a.b1[i], j.b, b_rows, b_cols, 1))) ||
            !make_tile_map(&a.b[i], j.b, b_rows, b_cols, 64) ||
            (!j.rows_on_n && !(j.out_f32 ? make_tile_map_f32(&a.out[i], j.out, out_rows, static_cast<uint64_t>(j.N), 32)
                        : make_tile_map(&a.out[i], j.out, out_rows, static_cast<uint64_t>(j.N), 32))))
            return cudaErrorInvalidValue;
        shallow |= j.by_rows && j.k_blocks <= kWideBlocks;
        units += product_units(j, E, cap);
        // as many as there are with rows spread evenly
        live += j.by_rows ? (tiles_of(cap) > E ? tiles_of(cap) : (cap < E ? cap : E)) * tiles_of(j.N)
                          : product_units(j, E, cap);
    }
    a.jobs = n;
    a.offsets = rows.offsets;
    a.num_rows = rows.num_rows;
    a.segment_rows = rows.segment_rows;
    a.E = E;
    a.cap = cap;
    a.err = err;
    a.wait_limit_ns = kWaitLimitNs;
    if (live <= kWideUnits * (num_sms / 2) || cap <= static_cast<long long>(kWideRows) * E || shallow)
        return launch_pair<WideConfig>(products_kernel<WideConfig>, a, units, num_sms, stream);
    return launch_pair<DeepConfig>(products_kernel<DeepConfig>, a, units, num_sms, stream);
}

cudaError_t launch_act_grad(const void *x, const void *dy, const void *W13, const void *W2, const int32_t *offsets,
                            int E, int cap, int H, int I, void *act, void *dgu, int32_t *err, int num_sms,
                            cudaStream_t stream)
{
    ActArgs a = {};
    const uint64_t rows = cap, h = H, i = I, e = E;
    if (!make_tile_map(&a.x, x, rows, h, 128) || !make_tile_map(&a.dy, dy, rows, h, 128) ||
        !make_tile_map(&a.x32, x, rows, h, kRowBox) || !make_tile_map(&a.dy32, dy, rows, h, kRowBox) ||
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
    const long long nt = (I + 127) / 128;
    if (cap <= static_cast<long long>(kSplitRows) * E) {
        if (!make_tile_map(&a.x64, x, rows, h, 64) || !make_tile_map(&a.dy64, dy, rows, h, 64) ||
            !make_tile_map(&a.w2_two, W2, e * h, i, 128))
            return cudaErrorInvalidValue;
        return launch_pair<SplitConfig>(act_grad_kernel<SplitConfig>, a, (tiles_of(cap) + E) * nt, num_sms, stream);
    }
    return launch_pair<ActConfig>(act_grad_kernel<ActConfig>, a, (tiles_of(cap) + E) * nt, num_sms, stream);
}

}  // namespace moe
