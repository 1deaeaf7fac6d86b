// route.cu -- the router: logits of every expert, scores, and the k experts
// of the largest keys with their weights.
//
//   logits[t, e] = sum_m x[t, m] w[e, m]        (x = h * r(h) * w_pre in moe_layer)
//
// Few tokens (moe_route up to 192, moe_layer): the router's weights are the bytes that matter
// (5.5 MB at E=384, H=7168) and must come from every SM at once, so a unit is
// 16 experts x a slice of H, about one unit per SM, and the slices' partial
// logits meet in the workspace. For one or two tokens the last CTA to get
// there (a count, nobody waits) sums them in slice order and selects, in the
// same kernel; for more a second kernel does, one CTA per token, launched
// early behind the first. (One cooperative kernel whose CTAs waited for all
// others at a grid-wide count took 8.1 us for one token and 2.3 us more when
// not in a graph: 2 us of it at the count, the rest the cooperative launch.)
// For moe_layer these kernels also write the experts' rows and, in the joined
// kernel, dispatch up to 32 routed slots, so that the expert kernel comes next.
// Products run on mma.sync m16n8k16 with the experts on M and 8 tokens on N:
// at these sizes the tensor work is nothing, and fragments taken straight
// from global memory need no staging. A dot product may take its terms in any
// order, so each thread loads 16 consecutive bytes of a row and calls them
// its fragment's K positions, for weights and tokens alike: every load is 16
// bytes and nothing is permuted.
//
// More tokens: logits on the tensor cores (route_gemm.cu), then a warp per
// token selects. (Selecting inside that kernel, a warp per token from the rows
// in shared memory, measured no better: T=8192, E=128 24.0 against 23.0 us,
// since there only 16 warps per SM are left to hide its latency.)
//
// In moe_layer the token operand is u = h * w_pre without r(h), which the sum
// does not need before its end: logits = r * sum u w. u is split exactly into
// bf16 parts (two when both factors are bf16: their product has 16 bits; three
// parts, 24 bits, otherwise), one MMA each, so the router sees the normalised
// row unrounded and no CTA waits for r.
#include <cuda_bf16.h>

#include "moe_internal.h"
#include "ptx.cuh"
#include "route_select.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------ many tokens

constexpr int kSelectWarps = 4;
constexpr int kDryBlocks = 608;

// One instance per 128, 256, 512 or 1024 experts: with the registers of the
// largest only a few warps fit on an SM.
template <int kPer>
__global__ void __launch_bounds__(32 * kSelectWarps) select_kernel(const __grid_constant__ RouteArgs a,
                                                                   const float *logits)
{
    extern __shared__ float s_keys[];   // [kSelectWarps][E], with groups only
    __shared__ SelectWarp s_warp[kSelectWarps];
    __shared__ float s_dry[32 * kPer];
    const int warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kSelectWarps + warp;
    // The first blocks sit on the SMs while the logits are still computed: they
    // run once over made-up logits (falling, so that few reach the bound) and
    // store nothing, which brings the code into the instruction caches (T=2048,
    // E=384 22.9 against 24.2 us; T=8192, E=128, where most blocks come later,
    // 24.8 against 24.9).
    const bool early = a.k <= 32 && blockIdx.x < kDryBlocks;
    for (int i = threadIdx.x; early && i < 32 * kPer; i += 32 * kSelectWarps)
        s_dry[i] = -0.125f * i;
    __syncthreads();
#pragma unroll 1
    for (int pass = early ? 0 : 1; pass < 2; ++pass) {
        if (pass == 1) {
            pdl_wait();
            pdl_trigger();
            if (t >= token_count(a.d_num_tokens, a.T_max))
                break;
        }
        const float *l = pass == 0 ? s_dry : logits + static_cast<size_t>(t) * a.E;
        select_token<kPer>(a, t, l, s_keys + warp * a.E, s_warp[warp], pass == 1);
        __syncwarp();
    }
}

template <int kPer>
cudaError_t launch_select(const RouteArgs &a, const float *logits, cudaStream_t stream, bool pdl)
{
    return launch_k(select_kernel<kPer>, dim3((a.T_max + kSelectWarps - 1) / kSelectWarps), dim3(32 * kSelectWarps),
                    a.n_group > 1 ? sizeof(float) * kSelectWarps * a.E : 0, stream, pdl, a, logits);
}

// ------------------------------------------------------------- few tokens

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t u)
{
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Eight consecutive values of a bf16 or fp32 row, as loaded.
struct Raw8 {
    uint4 a, b;       // b: fp32 only
};

__device__ __forceinline__ Raw8 load_raw8(const void *p, bool f32, size_t i)
{
    Raw8 r;
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + i * (f32 ? 4 : 2));
    r.a = __ldg(q);
    r.b = f32 ? __ldg(q + 1) : make_uint4(0u, 0u, 0u, 0u);
    return r;
}

__device__ __forceinline__ void widen8(const Raw8 &r, bool f32, float (&f)[8])
{
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 g = unpack_bf16(u[j]);
        f[2 * j] = f32 ? __uint_as_float(u[2 * j]) : g.x;
        f[2 * j + 1] = f32 ? __uint_as_float(u[2 * j + 1]) : g.y;
    }
}
// w' of the norm: 1, w or 1 + w
__device__ __forceinline__ void weight8(const RouteArgs &a, const Raw8 &r, float (&w)[8])
{
    if (!a.w_pre) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = 1.f;
        return;
    }
    widen8(r, a.w_f32, w);
    if (a.unit_offset)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = 1.f + w[i];
}

__device__ __forceinline__ Raw8 load_weight_raw8(const RouteArgs &a, int m)
{
    return a.w_pre ? load_raw8(a.w_pre, a.w_f32, m) : Raw8{};
}

// Shared memory of one selection by a whole block.
struct SelectScratch {
    float logits[kMaxExperts];
    uint32_t key[kMaxExperts];
    uint64_t found[kFewWarps * kMaxTopK];   // each warp's best, key and ~expert
    float warp[kFewWarps];
    float group[32];
    unsigned kept;
    float mx, sum;                          // softmax, where it is needed
    int id[kMaxTopK];
};

// All eight warps select for one token, logits in s.logits: each warp takes
// the k best of an eighth of the experts, then every one of those 8 k counts
// the ones that beat it. Called with a cold instruction cache between a
// model's other kernels, so its loops stay rolled: the version that one warp
// ran on unrolled registers took 13 us there.
//
// Leaves the ids in s.id; store_block then writes ids and weights (one warp).
__device__ void select_block(const RouteArgs &a, SelectScratch &s)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = a.E, k = a.k;
    bool bad = false;
    float mx = -INFINITY, sum = 1.f;
    for (int e = tid; e < E; e += kFewThreads) {
        float v = s.logits[e];
        if (!(v < INFINITY)) {   // NaN or +inf
            bad = true;
            s.logits[e] = v = -INFINITY;
        }
        mx = fmaxf(mx, v);
    }
    if (bad)
        atomicOr(a.err, MOE_DEVERR_BAD_LOGIT);
    if (needs_softmax(a)) {
        mx = warp_max(mx);
        if (lane == 0)
            s.warp[warp] = mx;
        __syncthreads();
        for (int i = 0; i < kFewWarps; ++i)
            mx = fmaxf(mx, s.warp[i]);
        mx = mx > -INFINITY ? mx : 0.f;
        sum = 0.f;
        for (int e = tid; e < E; e += kFewThreads)
            sum += expf(s.logits[e] - mx);
        sum = warp_sum(sum);
        __syncthreads();
        if (lane == 0)
            s.warp[warp] = sum;
        __syncthreads();
        sum = 0.f;
        for (int i = 0; i < kFewWarps; ++i)
            sum += s.warp[i];
    }
    for (int e = tid; e < E; e += kFewThreads)
        s.key[e] = order_key(key_float(a, e, s.logits[e], mx, sum));
    if (a.n_group > 1) {
        const int gs = E / a.n_group;
        __syncthreads();
        for (int g = warp; g < a.n_group; g += kFewWarps) {
            uint32_t first = 0u, second = 0u;
            for (int i = lane; i < gs; i += 32) {
                const uint32_t u = s.key[g * gs + i];
                second = u > first ? first : (u > second ? u : second);
                first = u > first ? u : first;
            }
            const uint32_t top = __reduce_max_sync(kFull, first);
            const int holder = __ffs(__ballot_sync(kFull, first == top)) - 1;
            const uint32_t next = __reduce_max_sync(kFull, lane == holder ? second : first);
            if (lane == 0)
                s.group[g] = top == 0u                            ? -INFINITY
                             : a.group_top == 1                   ? key_value(top)
                             : next == 0u                         ? -INFINITY
                                                                  : key_value(top) + key_value(next);
        }
        __syncthreads();
        if (warp == 0) {
            const unsigned kept = keep_groups(a, lane < a.n_group ? s.group[lane] : -INFINITY);
            if (lane == 0)
                s.kept = kept;
        }
        __syncthreads();
        for (int e = tid; e < E; e += kFewThreads)
            if (!((s.kept >> (e / gs)) & 1u))
                s.key[e] = 0u;
    }
    if (tid < kMaxTopK)
        s.id[tid] = -1;
    // this warp's best, over its own threads' experts (tid, tid + 256, ...)
    uint32_t key[kMaxExperts / kFewThreads];
#pragma unroll
    for (int i = 0; i < kMaxExperts / kFewThreads; ++i)
        key[i] = tid + i * kFewThreads < E ? s.key[tid + i * kFewThreads] : 0u;
    int n = 0;
#pragma unroll 1
    for (; n < k; ++n) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kMaxExperts / kFewThreads; ++i)
            if (key[i] > best) {
                best = key[i];
                at = tid + i * kFewThreads;
            }
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == 0u)
            break;
        const int e = __reduce_min_sync(kFull, best == top ? at : 1 << 30);
#pragma unroll
        for (int i = 0; i < kMaxExperts / kFewThreads; ++i)
            if (tid + i * kFewThreads == e)
                key[i] = 0u;
        if (lane == 0)
            s.found[warp * k + n] = static_cast<uint64_t>(top) << 32 | static_cast<uint32_t>(~e);
    }
    for (int i = lane; i < k; i += 32)
        if (i >= n)
            s.found[warp * k + i] = 0u;
    __syncthreads();
    for (int c = tid; c < kFewWarps * k; c += kFewThreads) {
        const uint64_t mine = s.found[c];
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < kFewWarps * k; ++i)
            rank += s.found[i] > mine ? 1 : 0;
        if (mine != 0u && rank < k)
            s.id[rank] = static_cast<int>(~static_cast<uint32_t>(mine));
    }
    if (tid == 0) {
        s.mx = mx;
        s.sum = sum;
    }
    __syncthreads();
}

__device__ void store_block(const RouteArgs &a, int t, const SelectScratch &s)
{
    const int lane = threadIdx.x & 31;
    int id[2];
    const int place[2] = {lane, lane + 32};
    float l[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        id[q] = s.id[lane + 32 * q];
        l[q] = id[q] >= 0 ? s.logits[id[q]] : -INFINITY;
    }
    const int n = __popc(__ballot_sync(kFull, id[0] >= 0)) + __popc(__ballot_sync(kFull, id[1] >= 0));
    store_choice(a, t, id, place, l, n, s.mx, s.sum);
}

// r(h) of a token, from the slices' sums of squares in slice order. The loads
// go out eight at a time: one after the other they cost 0.4 us each.
__device__ __forceinline__ float row_scale(const RouteArgs &a, const RouteSplit &sp, int t)
{
    const float *sq = a.part + static_cast<size_t>(sp.slices) * a.T_max * a.E + t;
    float sum = 0.f;
    for (int i0 = 0; i0 < sp.slices; i0 += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i0 + i < sp.slices ? __ldcg(sq + static_cast<size_t>(i0 + i) * a.T_max) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum += v[i];
    }
    return 1.f / sqrtf(sum / a.H + a.eps);
}

// Sum of one token's partial logits in slice order, times r(h) in moe_layer,
// into s.logits. Returns r.
template <bool kNormed>
__device__ __forceinline__ float gather_logits(const RouteArgs &a, const RouteSplit &sp, int t, SelectScratch &s)
{
    const int E = a.E;
    constexpr int kEach = kMaxExperts / kFewThreads;
    float sum[kEach] = {};
    for (int i0 = 0; i0 < sp.slices; i0 += 8) {
        float v[kEach][8];
#pragma unroll
        for (int j = 0; j < kEach; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = threadIdx.x + j * kFewThreads;
                v[j][i] = e < E && i0 + i < sp.slices
                              ? __ldcg(a.part + (static_cast<size_t>(i0 + i) * a.T_max + t) * E + e)
                              : 0.f;
            }
#pragma unroll
        for (int j = 0; j < kEach; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[j] += v[j][i];
    }
    const float r = kNormed ? row_scale(a, sp, t) : 1.f;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int e = threadIdx.x + j * kFewThreads;
        if (e < E) {
            s.logits[e] = sum[j] * r;
            if (a.logits)
                a.logits[static_cast<size_t>(t) * E + e] = sum[j] * r;
        }
    }
    __syncthreads();
    return r;
}

// The normalised row for the experts as two bf16 rows (bf16 is their MMAs'
// operand type): the leading parts and the rest, 16 bits together.
__device__ __forceinline__ void write_row(const RouteArgs &a, int t, float r)
{
    for (int m0 = 8 * threadIdx.x; m0 < a.H; m0 += 4 * 8 * kFewThreads) {
        Raw8 x[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + i * 8 * kFewThreads;
            if (m < a.H) {
                x[i] = load_raw8(a.x, a.x_f32, t * a.x_stride + m);
                w[i] = load_weight_raw8(a, m);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + i * 8 * kFewThreads;
            if (m >= a.H)
                break;
            float f[8], wp[8];
            widen8(x[i], a.x_f32, f);
            weight8(a, w[i], wp);
            uint32_t lead[4], rest[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float lo = f[2 * j] * r * wp[2 * j], hi = f[2 * j + 1] * r * wp[2 * j + 1];
                lead[j] = pack_bf16(lo, hi);
                const float2 taken = unpack_bf16(lead[j]);
                rest[j] = pack_bf16(lo - taken.x, hi - taken.y);
            }
            uint4 *const o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.x_out) +
                                                       2 * static_cast<size_t>(t) * a.H + m);
            o[0] = make_uint4(lead[0], lead[1], lead[2], lead[3]);
            o[a.H / 8] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
        }
    }
}

// The tables of moe_dispatch for R <= kRouteDispatchSlots slots, by one block:
// a slot's row is the count of the slots before it in (expert, slot) order.
// Threads first..kFewThreads - 1 of the block take part.
__device__ void dispatch_slots(const RouteArgs &a, const int *s_ids, int R, int first)
{
    const int tid = static_cast<int>(threadIdx.x) - first;
    if (tid < 0)
        return;
    for (int s = tid; s < R; s += kFewThreads - first) {
        const int e = s_ids[s];
        int row = 0;
#pragma unroll 4
        for (int j = 0; j < R; ++j) {
            const int o = s_ids[j];
            row += o >= 0 && (o < e || (o == e && j < s)) ? 1 : 0;
        }
        a.inv[s] = e >= 0 ? row : -1;
        if (e >= 0)
            a.perm[row] = s;
    }
    for (int e = tid; e <= a.E; e += kFewThreads - first) {
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < R; ++j)
            before += s_ids[j] >= 0 && s_ids[j] < e ? 1 : 0;
        a.expert_offsets[e] = before;
    }
}

// kTiles: 8-token tiles of a unit. kParts: bf16 parts of the token operand;
// 1: x as it is (moe_route), 2 or 3: u = h * w_pre (moe_layer).
template <int kTiles, int kParts>
__global__ void __launch_bounds__(kFewThreads, 1) route_few_kernel(const __grid_constant__ RouteArgs a,
                                                                   const RouteSplit sp)
{
    constexpr int kTok = 8 * kTiles;
    constexpr bool kJoin = kTiles == 1;    // the last CTA may select here (sp.join)
    __shared__ float s_acc[kFewWarps][16][kTok + 1];
    __shared__ float s_sq[kFewWarps][kTok];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int E = a.E, H = a.H;
    const int units = sp.groups * sp.slices * sp.chunks;
    const int blocks64 = H / 64;
    const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(a.w);
    // this CTA's weights on their way into L2 before the wait for the
    // previous kernel (a prefetch reads nothing that kernel could still write)
    {
        const int u = blockIdx.x;
        const int e0 = (u % sp.groups) * 16, s = (u / sp.groups) % sp.slices;
        const int m0 = 64 * (s * blocks64 / sp.slices), m1 = 64 * ((s + 1) * blocks64 / sp.slices);
        const int lines = (m1 - m0) / 64;    // of 128 bytes, per row
        for (int i = threadIdx.x; i < 16 * lines; i += kFewThreads)
            if (e0 + i / lines < E)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(w + static_cast<size_t>(e0 + i / lines) * H + m0 +
                                                              64 * (i % lines)));
    }
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a.d_num_tokens, a.T_max);

    const int t0 = static_cast<int>(blockIdx.x) / sp.groups / sp.slices * kTok;
    if (t0 < T) {
        const int u = blockIdx.x;
        const int e0 = (u % sp.groups) * 16, s = (u / sp.groups) % sp.slices;
        const int b0 = 2 * (s * blocks64 / sp.slices), b1 = 2 * ((s + 1) * blocks64 / sp.slices);   // 32-wide blocks
        float acc[kTiles][4] = {};
        float sq[kTiles] = {};
        const bool lo_row = e0 + g < E, hi_row = e0 + g + 8 < E;
        const uint4 *w_lo = reinterpret_cast<const uint4 *>(w + static_cast<size_t>(e0 + g) * H + 8 * q);
        const uint4 *w_hi = reinterpret_cast<const uint4 *>(w + static_cast<size_t>(e0 + g + 8) * H + 8 * q);
        const bool squares = kParts > 1 && e0 == 0;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        // K blocks of a warp in flight, weights and tokens: five cover a slice of
        // the decode workloads (E=384, H=7168) in one round trip
        constexpr int kAhead = kTiles == 1 ? 5 : (kTiles == 2 ? 3 : 2);
        for (int bb = b0 + warp; bb < b1; bb += kAhead * kFewWarps) {
            uint4 wl[kAhead], wh[kAhead];
            Raw8 x[kAhead][kTiles], wr[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int b = bb + i * kFewWarps;
                const int m = 32 * b + 8 * q;
                wl[i] = (b < b1 && lo_row) ? __ldg(w_lo + 4 * b) : zero;
                wh[i] = (b < b1 && hi_row) ? __ldg(w_hi + 4 * b) : zero;
                wr[i] = kParts > 1 && b < b1 ? load_weight_raw8(a, m) : Raw8{};
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    const int t = t0 + 8 * j + g;
                    x[i][j] = b < b1 && t < T ? load_raw8(a.x, kParts > 1 && a.x_f32, t * a.x_stride + m) : Raw8{};
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (bb + i * kFewWarps >= b1)
                    break;
                float wp[8];
                if (kParts > 1)
                    weight8(a, wr[i], wp);
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    if (kParts == 1) {
                        const uint4 xv = x[i][j].a;
                        mma_bf16(acc[j], wl[i].x, wh[i].x, wl[i].y, wh[i].y, xv.x, xv.y);
                        mma_bf16(acc[j], wl[i].z, wh[i].z, wl[i].w, wh[i].w, xv.z, xv.w);
                    } else {
                        float f[8];
                        widen8(x[i][j], a.x_f32, f);
                        if (squares)
#pragma unroll
                            for (int v = 0; v < 8; ++v)
                                sq[j] = fmaf(f[v], f[v], sq[j]);
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            f[v] *= wp[v];
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            uint32_t p[4];
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                p[v] = pack_bf16(f[2 * v], f[2 * v + 1]);
                                const float2 taken = unpack_bf16(p[v]);
                                f[2 * v] -= taken.x;
                                f[2 * v + 1] -= taken.y;
                            }
                            mma_bf16(acc[j], wl[i].x, wh[i].x, wl[i].y, wh[i].y, p[0], p[1]);
                            mma_bf16(acc[j], wl[i].z, wh[i].z, wl[i].w, wh[i].w, p[2], p[3]);
                        }
                    }
                }
            }
        }
        // the warps' sums (rows g and g + 8, tokens 2q and 2q + 1 of each tile) meet in shared memory
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            s_acc[warp][g][8 * j + 2 * q] = acc[j][0];
            s_acc[warp][g][8 * j + 2 * q + 1] = acc[j][1];
            s_acc[warp][g + 8][8 * j + 2 * q] = acc[j][2];
            s_acc[warp][g + 8][8 * j + 2 * q + 1] = acc[j][3];
            if (squares) {
                float v = sq[j];
                v += __shfl_xor_sync(kFull, v, 1);
                v += __shfl_xor_sync(kFull, v, 2);
                if (q == 0)
                    s_sq[warp][8 * j + g] = v;
            }
        }
        __syncthreads();
        float *part = a.part + static_cast<size_t>(s) * a.T_max * E;
        for (int i = threadIdx.x; i < 16 * kTok; i += kFewThreads) {
            const int r = i & 15, c = i >> 4;
            if (e0 + r < E && t0 + c < T) {
                float v = 0.f;
#pragma unroll
                for (int x = 0; x < kFewWarps; ++x)
                    v += s_acc[x][r][c];
                part[static_cast<size_t>(t0 + c) * E + e0 + r] = v;
            }
        }
        if (squares)
            for (int c = threadIdx.x; c < kTok; c += kFewThreads)
                if (t0 + c < T) {
                    float v = 0.f;
                    for (int x = 0; x < kFewWarps; ++x)
                        v += s_sq[x][c];
                    a.part[static_cast<size_t>(sp.slices) * a.T_max * E + static_cast<size_t>(s) * a.T_max + t0 + c] = v;
                }
        __syncthreads();
    }

    if constexpr (kJoin) {
        if (!sp.join)
            return;
        __shared__ SelectScratch s_sel;
        __shared__ int s_ids[kRouteDispatchSlots];
        __shared__ int s_last;
        if (kParts > 1)       // the rows and w_pre into L1: the last CTA, whichever it is, writes the rows
            for (int m = 32 * threadIdx.x; m < H; m += 32 * kFewThreads) {
                for (int t = 0; t < T; ++t)
                    prefetch_l1(static_cast<const char *>(a.x) + (t * a.x_stride + m) * (a.x_f32 ? 4 : 2));
                if (a.w_pre)
                    prefetch_l1(static_cast<const char *>(a.w_pre) + m * (a.w_f32 ? 4 : 2));
            }
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0)
            s_last = atom_add_acq_rel_gpu(a.counters, 1) == units - 1;
        __syncthreads();
        if (!s_last)
            return;
        if (threadIdx.x == 0)
            *a.counters = 0;
        for (int t = 0; t < T; ++t) {
            const float r = gather_logits<(kParts > 1)>(a, sp, t, s_sel);
            if (kParts > 1)
                write_row(a, t, r);
            select_block(a, s_sel);
            if (a.perm) {
                for (int j = threadIdx.x; j < a.k; j += kFewThreads)
                    s_ids[t * a.k + j] = s_sel.id[j];
                __syncthreads();
            }
            if (warp == 0)
                store_block(a, t, s_sel);
            else if (a.perm && t == T - 1)
                dispatch_slots(a, s_ids, T * a.k, 32);
            if (t < T - 1)
                __syncthreads();
        }
        if (a.perm && T == 0)
            dispatch_slots(a, s_ids, 0, 0);
    }
}

// What follows the partial logits of more than two tokens: CTA t selects for
// token t, CTA T_max + t writes its rows for the experts (moe_layer). (The last
// CTA that selected dispatching as well, as the joined kernel's does, measured
// slower than a dispatch kernel behind this one from 24 slots on: 39.1 against
// 38.2 us a layer, 59.7 against 55.9 at 128 slots.)
template <bool kNormed>
__global__ void __launch_bounds__(kFewThreads) route_finish_kernel(const __grid_constant__ RouteArgs a,
                                                                   const RouteSplit sp)
{
    __shared__ SelectScratch s_sel;
    pdl_wait();
    pdl_trigger();
    const int T = token_count(a.d_num_tokens, a.T_max);
    const int job = blockIdx.x;
    if (job >= a.T_max) {
        const int t = job - a.T_max;
        if (kNormed && t < T)
            write_row(a, t, row_scale(a, sp, t));
        return;
    }
    if (job < T) {
        gather_logits<kNormed>(a, sp, job, s_sel);
        select_block(a, s_sel);
        if (threadIdx.x < 32)
            store_block(a, job, s_sel);
    }
}

template <int kTiles>
cudaError_t launch_few(const RouteArgs &a, const RouteSplit &sp, cudaStream_t stream, bool pdl)
{
    const bool exact16 = !a.x_f32 && !a.unit_offset && (!a.w_pre || !a.w_f32);
    auto kern = exact16 ? route_few_kernel<kTiles, 2> : route_few_kernel<kTiles, 3>;
    if (!a.normed)
        kern = route_few_kernel<kTiles, 1>;
    const cudaError_t e =
        launch_k(kern, dim3(sp.groups * sp.slices * sp.chunks), dim3(kFewThreads), 0, stream, pdl, a, sp);
    if (e != cudaSuccess || sp.join)
        return e;
    return a.normed ? launch_k(route_finish_kernel<true>, dim3(2 * a.T_max), dim3(kFewThreads), 0, stream, pdl, a, sp)
                    : launch_k(route_finish_kernel<false>, dim3(a.T_max), dim3(kFewThreads), 0, stream, pdl, a, sp);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream, bool pdl)
{
    if (a.normed || a.T_max <= kRouteFewTokens) {
        const RouteSplit sp = route_split(a.T_max, a.E, a.H, a.one_kernel != 0);
        switch (sp.tiles) {
        case 1:
            return launch_few<1>(a, sp, stream, pdl);
        case 2:
            return launch_few<2>(a, sp, stream, pdl);
        default:
            return launch_few<4>(a, sp, stream, pdl);
        }
    }
    float *logits = a.logits ? a.logits : a.part;
    const cudaError_t e = launch_route_gemm(a, logits, stream, pdl);
    if (e != cudaSuccess)
        return e;
    if (a.E <= 128)
        return launch_select<4>(a, logits, stream, pdl);
    if (a.E <= 256)
        return launch_select<8>(a, logits, stream, pdl);
    if (a.E <= 512)
        return launch_select<16>(a, logits, stream, pdl);
    return launch_select<32>(a, logits, stream, pdl);
}

}  // namespace moe
