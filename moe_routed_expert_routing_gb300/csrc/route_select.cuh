// route_select.cuh -- the router's selection by one warp: scores, groups, the k
// experts of the largest keys and their weights, from one token's logits.
#pragma once

#include <cfloat>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int token_count(const int32_t *d_num_tokens, int T_max)
{
    int T = T_max;
    if (d_num_tokens) {
        T = *d_num_tokens;
        T = T < 0 ? 0 : (T > T_max ? T_max : T);
    }
    return T;
}

// A float as an unsigned integer of the same order; 0 for what may not be
// chosen (-inf and NaN). -0 and +0 give the same number.
__device__ __forceinline__ uint32_t order_key(float f)
{
    f = f + 0.f;
    const uint32_t b = __float_as_uint(f);
    const uint32_t u = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return f > -INFINITY ? u : 0u;   // false for NaN too
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

__device__ __forceinline__ float score_of(const RouteArgs &a, float l, float mx, float sum)
{
    return a.sigmoid ? 1.f / (1.f + expf(-l)) : expf(l - mx) / sum;
}

// Float of an order_key (which is not 0).
__device__ __forceinline__ float key_value(uint32_t u)
{
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// log of the sigmoid, without overflow or a loss of small values
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.f) - log1pf(expf(-fabsf(l))); }

// The key an expert is chosen by, 0 if it may not be; l is its logit (finite
// or -inf), mx and sum the softmax's maximum and denominator.
__device__ __forceinline__ bool keyed_by_score(const RouteArgs &a) { return a.bias != nullptr || a.group_top > 1; }

__device__ __forceinline__ float key_float(const RouteArgs &a, int e, float l, float mx, float sum)
{
    if (keyed_by_score(a) && l > -INFINITY)
        return score_of(a, l, mx, sum) + (a.bias ? __ldg(a.bias + e) : 0.f);
    return l;
}

// The softmax over all experts is needed only where a key or a weight is a
// score; renormalised weights need the chosen logits alone.
__device__ __forceinline__ bool needs_softmax(const RouteArgs &a)
{
    return !a.sigmoid && (keyed_by_score(a) || !a.renormalize);
}

// The chosen experts' ids and weights, by one warp: a lane holds up to two of
// them (id -1: none) with their places. n: how many were found; places from n
// on get id -1 and weight 0.
__device__ __forceinline__ void store_choice(const RouteArgs &a, int t, const int (&id)[2], const int (&place)[2],
                                             const float (&l)[2], int n, float mx, float sum, bool store = true)
{
    float w[2], norm = 1.f;
    if (a.renormalize) {
        // the chosen scores over their sum, from their logarithms (the softmax
        // over all E cancels), so that scores that underflow keep their ratios
        float lg[2], top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            lg[q] = id[q] >= 0 ? (a.sigmoid ? log_sigmoid(l[q]) : l[q]) : -INFINITY;
            top = fmaxf(top, lg[q]);
        }
        const uint32_t high = __reduce_max_sync(kFull, order_key(top));
        top = high ? key_value(high) : 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w[q] = expf(lg[q] - top);
        norm = warp_sum(w[0] + w[1]);
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w[q] = id[q] >= 0 ? score_of(a, l[q], mx, sum) : 0.f;
    }
    if (!store)
        return;
    int32_t *ids = a.ids + static_cast<size_t>(t) * a.k;
    float *weights = a.weights + static_cast<size_t>(t) * a.k;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (id[q] >= 0) {
            ids[place[q]] = id[q];
            weights[place[q]] = a.scale * __fdividef(w[q], norm);   // norm in [1, 64]: within two units
        }
    for (int j = n + (threadIdx.x & 31); j < a.k; j += 32) {
        ids[j] = -1;
        weights[j] = 0.f;
    }
}

// Which groups stay, from lane g's group value: bit g of the result. One warp.
__device__ __forceinline__ unsigned keep_groups(const RouteArgs &a, float value)
{
    const int lane = threadIdx.x & 31;
    if (!(value > -INFINITY))   // also the sum of +inf and -inf
        value = -INFINITY;
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
        const float o = __shfl_sync(kFull, value, g);
        rank += (o > value || (o == value && g < lane)) ? 1 : 0;
    }
    return __ballot_sync(kFull, lane < a.n_group && rank < a.topk_group);
}

// The groups that stay, from one token's keys in shared memory (-inf: none).
// One warp: 32 / n_group lanes take a group.
__device__ __noinline__ unsigned kept_groups(const RouteArgs &a, const float *s_key)
{
    const int lane = threadIdx.x & 31, gs = a.E / a.n_group, per = 32 / a.n_group;
    const int g = lane / per, part = lane % per;
    float first = -INFINITY, second = -INFINITY;
    if (g < a.n_group)
        for (int i = part; i < gs; i += per) {
            const float v = s_key[g * gs + i];
            second = fmaxf(second, fminf(first, v));
            first = fmaxf(first, v);
        }
    float top1 = first, top2 = second;       // of the group's first lane
    for (int j = 1; j < per; ++j) {
        const float f = __shfl_down_sync(kFull, first, j), s = __shfl_down_sync(kFull, second, j);
        top2 = fmaxf(fmaxf(top2, s), fminf(top1, f));
        top1 = fmaxf(top1, f);
    }
    const float value = a.group_top > 1 ? top1 + top2 : top1;
    return keep_groups(a, __shfl_sync(kFull, value, lane * per));
}

// k rounds of a warp-wide maximum, each below the last: for k > 32, and for
// rows with many equal keys. kept: bit g set if group g stays.
__device__ __noinline__ void select_by_rounds(const RouteArgs &a, int t, const float *logits, unsigned kept, float mx,
                                              float sum)
{
    const int lane = threadIdx.x & 31, gs = a.E / a.n_group;
    int id0 = -1, id1 = -1, n = 0;
    uint64_t last = ~0ull;
    for (; n < a.k; ++n) {
        uint64_t best = 0;
        for (int e = lane; e < a.E; e += 32) {
            const float l = logits[e];
            if (!(l < INFINITY) || !((kept >> (e / gs)) & 1u))
                continue;
            const uint32_t u = order_key(key_float(a, e, l, mx, sum));
            const uint64_t c = static_cast<uint64_t>(u) << 32 | static_cast<uint32_t>(~e);
            if (u && c < last && c > best)
                best = c;
        }
        const uint32_t top = __reduce_max_sync(kFull, static_cast<uint32_t>(best >> 32));
        if (top == 0u)
            break;
        const uint32_t low =
            __reduce_max_sync(kFull, static_cast<uint32_t>(best >> 32) == top ? static_cast<uint32_t>(best) : 0u);
        last = static_cast<uint64_t>(top) << 32 | low;
        if (lane == (n & 31))
            (n < 32 ? id0 : id1) = static_cast<int>(~low);
    }
    const int id[2] = {id0, id1}, place[2] = {lane, lane + 32};
    const float l[2] = {id0 >= 0 ? logits[id0] : 0.f, id1 >= 0 ? logits[id1] : 0.f};
    store_choice(a, t, id, place, l, n, mx, sum);
}

// Shared memory of one warp's selection: the keys that reach the bound, with
// ~expert below them, so that the larger word is the better one.
struct __align__(8) SelectWarp {
    uint64_t found[32];
};

// One warp selects for one token whose logits lie in logits[E]; lane i holds
// experts i, i + 32, ... s_key: E floats of scratch, used with groups only.
// store: false for a run whose result is not wanted (see select_kernel).
//
// k rounds of a warp-wide maximum over all keys would be k passes over the
// lane's registers. k rounds over the lanes' own maxima give a lower bound of
// the k-th largest key instead, and few keys reach it (8 to 10 of 128 or 384
// at k = 6 to 8): those are gathered, and each counts the ones that beat it.
// The code is short on purpose: it runs once or twice per warp right after
// other code, and unrolled over four tokens it waited for instruction fetches
// (12,000 cycles for the four, no faster than one after the other).
template <int kPer>
__device__ __forceinline__ void select_token(const RouteArgs &a, int t, const float *logits, float *s_key, SelectWarp &s,
                                             bool store = true)
{
    const int lane = threadIdx.x & 31;
    float v[kPer];
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v[i] = lane + 32 * i < a.E ? logits[lane + 32 * i] : -INFINITY;
        total += v[i];
    }
    // NaN and +inf reach the total (as a sum past the range of fp32 does); -inf alone leaves it below
    if (__any_sync(kFull, !(total < INFINITY))) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (!(v[i] < INFINITY)) {
                bad = true;
                v[i] = -INFINITY;
            }
        if (bad)
            atomicOr(a.err, MOE_DEVERR_BAD_LOGIT);
    }
    float mx = 0.f, sum = 1.f;
    if (needs_softmax(a)) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            m = fmaxf(m, v[i]);
        const uint32_t high = __reduce_max_sync(kFull, order_key(m));
        mx = high ? key_value(high) : 0.f;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            sum += expf(v[i] - mx);
        sum = warp_sum(sum);
    }
    if (keyed_by_score(a))
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (v[i] > -INFINITY)
                v[i] = key_float(a, lane + 32 * i, v[i], mx, sum);
    unsigned kept = ~0u;
    if (a.n_group > 1) {
        const int gs = a.E / a.n_group;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < a.E)
                s_key[lane + 32 * i] = v[i] > -INFINITY ? v[i] : -INFINITY;   // NaN: none
        __syncwarp();
        kept = kept_groups(a, s_key);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i >= a.E || !((kept >> ((lane + 32 * i) / gs)) & 1u))
                v[i] = -INFINITY;
    }
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        best = fmaxf(best, v[i]);      // a NaN key is left out
    uint32_t own = order_key(best), least = 0u;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
        least = __reduce_max_sync(kFull, own);
        own = own == least ? 0u : own;   // equal lanes leave together: the bound is only lower
    }
    const float bound = least ? key_value(least) : -FLT_MAX;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool in = v[i] >= bound;
        const unsigned b = __ballot_sync(kFull, in);
        if (b == 0u)
            continue;
        const int slot = n + __popc(b & ((1u << lane) - 1u));
        if (in && slot < 32)
            s.found[slot] = static_cast<uint64_t>(order_key(v[i])) << 32 | static_cast<uint32_t>(~(lane + 32 * i));
        n += __popc(b);
    }
    if (n > 32 || a.k > 32) {
        if (store)
            select_by_rounds(a, t, logits, kept, mx, sum);
        return;
    }
    __syncwarp();
    const uint64_t mine = lane < n ? s.found[lane] : 0u;
    int rank = 0;
#pragma unroll 2
    for (int i = 0; i < n; ++i)
        rank += s.found[i] > mine ? 1 : 0;
    int id[2] = {-1, -1};
    const int place[2] = {rank, 0};
    float l[2] = {-INFINITY, -INFINITY};
    if (lane < n && rank < a.k) {
        id[0] = static_cast<int>(~static_cast<uint32_t>(mine));
        l[0] = keyed_by_score(a) ? logits[id[0]] : key_value(static_cast<uint32_t>(mine >> 32));
    }
    store_choice(a, t, id, place, l, min(n, a.k), mx, sum, store);
}

}  // namespace

}  // namespace moe
