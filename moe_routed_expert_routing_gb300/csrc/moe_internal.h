// moe_internal.h -- declarations shared by the translation units of libmoe.so
// (kernels + launchers). Not part of the public ABI (include/moe.h is).
#pragma once

#include <cstddef>
#include <cstdint>
#include <utility>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe.h"

namespace moe {

// ---- limits of this build (checked by host validation) ----
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kDispatchThreads = 256;
constexpr int kDispatchSlotsPerBlock = 1024;  // routed slots counted/scattered by one block

// Pipeline waits inside the GEMM kernels give up after this long (the device
// error word then carries MOE_DEVERR_WAIT_TIMEOUT).
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// ---- programmatic dependent launch ----
// With `pdl` set, a kernel of the library may start while the kernel before
// it on the stream is still finishing (cudaLaunchAttributeProgrammaticStream-
// Serialization): it runs its prologue, then waits (griddepcontrol.wait) for
// the previous grid's completion and memory before touching any global data
// (but for what a kernel two or more launches back wrote),
// and releases its own dependents (griddepcontrol.launch_dependents), only
// after that wait, by every thread: one thread's release counts for its block. Every
// kernel waits before it finishes, so completion stays
// transitive along the stream, and when a kernel starts, every kernel two or
// more launches back has completed; without the attribute both instructions
// are no-ops. The norms, the router and the gradients of both and of the experts use it; of the expert GEMMs'
// paths the host turns it on for the M-small (decode) one only: measured in one process, it saves
// ~8 us per decode step and costs ~90 us per large-batch step, where the early
// dependents share the SMs with the persistent GEMM.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l1(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

template <typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                     Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---- kernels whose CTAs wait on one another ----
// Such a kernel is correct only if every CTA of its grid is resident at
// once. The launch asks for that guarantee (cudaLaunchAttributeCooperative:
// the grid starts only when all of its CTAs fit, and a grid that could never
// fit is refused), and the host first sizes the grid against the occupancy
// the device reports for the kernel. Pure host arithmetic: the grid to
// launch for `want` CTAs when `per_sm` CTAs fit on one of `sms` SMs, or 0
// when none fits (the launch is then refused before it is made).
inline int coresident_grid(long long want, int per_sm, int sms)
{
    if (want < 1 || per_sm < 1 || sms < 1)
        return 0;
    const long long most = static_cast<long long>(per_sm) * sms;
    return static_cast<int>(want < most ? want : most);
}

// SMs the fused decode kernel's grid may use. The dispatch block launched
// before it and one of its CTAs cannot share an SM (shared memory), and the
// cooperative launch waits until the whole grid fits. Where its gate-up
// units (at most (min(cap, E) + cap / tile_rows) row tiles x ceil(I / 128))
// fit one wave on one SM fewer (a few tokens; bf16, three-kernel form) the
// grid leaves that SM to the dispatch, so the kernel starts, and runs its
// prologue, under it. Measured at one token, E=384, H=7168, I=3072, in one
// process, outputs bit-identical: 127.4 vs 128.3 us per call; at eight
// tokens the SM is worth more.
inline int fused_grid_sms(bool whole_forward, bool mxfp8, long long cap, int E, int I, int tile_rows, int sms)
{
    const long long tiles_bound = (cap < E ? cap : E) + cap / tile_rows;
    const long long units1_bound = tiles_bound * ((I + 127) / 128);
    return (!whole_forward && !mxfp8 && sms > 1 && units1_bound <= sms - 1) ? sms - 1 : sms;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_k_coresident(void (*kernel)(KArgs...), long long want_ctas, dim3 block, size_t smem,
                                cudaStream_t stream, bool pdl, int sms, Args &&...args)
{
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, static_cast<int>(block.x),
                                                                  smem);
    if (e != cudaSuccess)
        return e;
    const int grid = coresident_grid(want_ctas, per_sm, sms);
    if (grid < 1)
        return cudaErrorCooperativeLaunchTooLarge;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The norms around the block (norm.cu, combine_residual.cu, grouped_gemm.cu)
struct NormArgs {
    const void *h;             // residual stream, bf16 or fp32
    const void *y;             // block output, bf16 (null: norm of h only)
    const void *w_post;        // null: no weight
    const void *gate;
    const void *w_next;        // weight of x_next (moe_norm: of x); null: no weight
    const int32_t *d_num_tokens;
    void *h_out;
    void *x;                   // x_next (moe_norm: x), bf16; null: not computed
    int T_max, H;
    int h_f32, w_f32, unit_offset, norm_block, gate_kind;
    float eps, scale;
    long long h_stride, y_stride, x_stride, out_stride, gate_stride;
};

// ---- dispatch (dispatch.cu) ----
cudaError_t launch_dispatch(const int32_t *topk_ids, const int32_t *d_num_tokens, int T_max, int k, int E,
                            int32_t *block_counts, int32_t *block_base, int32_t *expert_offsets,
                            int32_t *perm, int32_t *inv, int32_t *err, cudaStream_t stream, bool pdl);

cudaError_t launch_gather_rows(const void *x, const int32_t *perm, const int32_t *expert_offsets, int E, int k,
                               int H, int cap, void *x_sorted, int num_sms, cudaStream_t stream, bool pdl,
                               int pair = 0);

// ---- combine (combine.cu) ----
// y_sorted is fp32, or fp16 when y_f16 is set (moe_forward's tiled paths).
// fp32 y may be `parts` partial buffers of a down GEMM that split K,
// part_stride elements apart: each row is their sum in part order.
// routing_early: inv was written at least two launches back on this stream
// (moe_forward) and the token count and weights are inputs, so the kernel
// may pull a block's routing into L1 before its dependency wait.
cudaError_t launch_combine(const void *y_sorted, bool y_f16, const int32_t *inv, const float *topk_weights,
                           const int32_t *d_num_tokens, int T_max, int k, int H, void *out, int num_sms,
                           cudaStream_t stream, bool pdl, int parts = 1, size_t part_stride = 0,
                           bool routing_early = false);

// y_sorted[r] = ((p0 + p1) + p2) + p3 over the `parts` fp32 partial buffers of
// [cap, H] starting at parts_base, for r < expert_offsets[E].
cudaError_t launch_reduce_parts(const float *parts_base, int parts, const int32_t *expert_offsets, int E, int H,
                                int cap, float *y_sorted, int num_sms, cudaStream_t stream, bool pdl);

// ---- packed weights (weights_pack.cu) ----
cudaError_t launch_pack_weights(const void *W13, const void *W2, void *W13_packed, void *W2_packed, int E, int H,
                                int I, int num_sms, cudaStream_t stream);

// ---- MXFP8 weights (weights_mx.cu) ----
// W13[E, 2I, H] and W2[E, H, I] bf16 -> the MOE_WEIGHTS_MXFP8 buffers: E4M3
// codes (row-major), then the E8M0 scale codes in (128-row tile, 128-wide K
// block, row, sub-block) order.
cudaError_t launch_quantize_weights_mxfp8(const void *W13, const void *W2, void *W13_mx, void *W2_mx, int E, int H,
                                          int I, int num_sms, cudaStream_t stream);

// ---- expert GEMMs (grouped_gemm.cu) ----
struct GemmProblem {
    const void *act;          // [act_rows, K] bf16: sorted rows, or x itself when gather is set
    int act_rows;             // rows of `act` (cap, or T_max for x)
    bool gather;              // A rows fetched from x through perm (tile::gather4), gate-up only
    const int32_t *perm;      // gather: sorted row -> routed slot
    int k;                    // gather: token = slot / k
    const void *w;            // [E, w_rows_per_expert, K] bf16
    void *out;                // [cap, n_out]: bf16 h (gated) or fp32 y (down)
    const int32_t *expert_offsets;
    int32_t *err;
    int E, cap, K, n_out;
    int w_rows_per_expert;
    int up_row_offset;        // gated: row offset of the up half inside one expert
    bool gated;               // fused SiLU(gate) * up epilogue
    bool small_m;             // weights on the MMA M side (M-small path)
    int tile_rows;            // activation rows per tile: 128 (tiled) or 16/32/64 (M-small)
    int split_k;              // 1, 2 or 4 (M-small down GEMM only): K parts, part p of fp32 out at out + p * cap * n_out
    bool pdl;                 // programmatic dependent launch
    bool cta_pair;            // tiled path on 2-CTA clusters (tcgen05 cta_group::2)
    bool w_packed;            // `w` is in the access-ordered PACKED layout
    bool w_mxfp8;             // `w` is in the MXFP8 layout (codes, then scale blocks): fused kernel only
    bool out_f16;             // tiled down GEMM: y as fp16 (saturated; MOE_DEVERR_Y_RANGE if clipped)
    int pair = 0;             // 1: paired rows (moe_layer; see GemmArgs)
    int32_t *sched = nullptr; // single-CTA grouped GEMM (M-small and tiled): two workspace counters (units
                              // handed out, CTAs at the tail), zero before the launch and left zero by it;
                              // null: units dealt round-robin
};

cudaError_t launch_grouped_gemm(const GemmProblem &p, int num_sms, cudaStream_t stream);

// The rest of moe_forward for the whole-forward form of the fused kernel:
// the dispatch inputs and outputs and the combine's weights and output.
struct MegaParams {
    const int32_t *ids;            // [T_max, k]
    const float *topk_w;           // [T_max, k]
    const int32_t *d_num_tokens;   // nullable
    int T_max;
    int32_t *expert_offsets_out;   // [E + 1]
    int32_t *perm_out;             // [cap]
    void *out;                     // [T_max, H] bf16
    // the dispatch kernel runs beside the fused kernel (and writes the tables
    // above and inv) and the combine kernel after it: the fused kernel only
    // dispatches locally for its own units
    bool combine_apart = false;
    // moe_layer: in place of the combine, the way back into the residual
    // stream (null: combine into `out`), with fp32 scratch for y [T_max, H]
    // and for row sums (tail_sum_floats)
    const NormArgs *tail = nullptr;
    float *tail_y = nullptr;
    float *tail_sums = nullptr;
};

inline size_t tail_sum_floats(int T_max, int H) { return 2 * static_cast<size_t>(T_max) * ((H + 1023) / 1024); }

// Both M-small GEMMs in one persistent launch (gate-up with gathered rows, then
// down). ready[E] and counters[2] must be zero when the kernel starts; the
// kernel leaves them at zero (the last CTA out clears them), so a workspace
// that starts zeroed needs no clearing between calls. With `mega`, the launch
// is the whole forward (dispatch, both GEMMs, combine); up.perm and the
// expert_offsets of both problems are then not read, and a split down GEMM
// writes its halves to down.out and down.out + cap * H (no zeroing needed).
cudaError_t launch_fused_small(const GemmProblem &up, const GemmProblem &down, int32_t *ready, int32_t *counters,
                               int num_sms, cudaStream_t stream, const MegaParams *mega = nullptr);

// Whether the whole-forward kernel's shared-memory expert tables for E experts
// and `slots` = T_max * k routed slots fit next to its pipeline on this device.
bool fused_mega_fits(int E, long long slots, bool mxfp8);

// ---- norms around the block (norm.cu) ----
// x = norm(h) (y null), or h_out = h + s * g * norm(y) and x = norm(h_out).
cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t stream, bool pdl);

// The end of moe_layer (combine_residual.cu): combine into an unrounded y, then
// as launch_norm with that y; y_sorted (of paired rows), inv (of routed rows)
// and parts as launch_combine takes them.
cudaError_t launch_combine_residual(const float *y_sorted, const int32_t *inv, const float *topk_weights,
                                    const NormArgs &a, int k, int parts, size_t part_stride, cudaStream_t stream,
                                    bool pdl);

// ---- router (route.cu) ----
struct RouteArgs {
    const void *x;             // [T_max, H] bf16; moe_layer: the residual stream, x_f32 of either type
    const void *w;             // [E, H] bf16
    const float *bias;         // null: none
    const int32_t *d_num_tokens;
    int32_t *ids;
    float *weights;
    float *logits;             // [T_max, E], or null: not wanted
    int32_t *err;
    int32_t *counters;         // one, zero at launch and at exit (few tokens)
    float *part;               // workspace, route_scratch_floats() of them
    int T_max, E, k, H;
    int sigmoid, renormalize, n_group, topk_group, group_top;
    float scale;
    // moe_layer: the router reads x * r(x) * w_pre before its rounding, and
    // writes the rounded rows to x_out
    int normed, x_f32, w_f32, unit_offset;
    const void *w_pre;         // null: no weight
    void *x_out;               // [2 * T_max, H] bf16: each row's leading part and the rest (paired rows)
    // moe_layer, joined kernel, at most kRouteDispatchSlots slots: moe_dispatch's tables, or null
    int32_t *expert_offsets, *perm, *inv;
    int one_kernel;            // the last CTA selects for up to 16 tokens, in the same kernel
    long long x_stride;
    float eps;
};

// The few-token kernel's split of [T_max, E, H]: units of 16 experts x one
// slice of H x up to 32 tokens, about one per SM. The narrowest units that
// leave H in four slices or more, else the widest: 32 tokens of E=128, H=4096
// 6.4 us in units of 8 tokens, 7.3 in one of 32; 24 tokens of E=384, H=7168
// 9.3 and 8.2; 61 of E=256, H=7168 11.9 and 9.4.
struct RouteSplit {
    int tiles;                 // 8-token tiles of a unit: 1, 2 or 4
    int chunks, groups, slices;
    bool join;                 // one kernel: its last CTA selects
};

// moe_route takes the few-token kernels up to here, then the tensor-core ones
// (route_gemm.cu). 128 tokens of E=128, H=4096 7.8 us against 10.2, 96 of E=256,
// H=7168 10.3 against 12.4, 190 of E=128 9.0 against 10.2; 256 of E=256 17.4
// against 12.5. moe_layer, whose router reads unrounded rows, takes them always.
constexpr int kRouteFewTokens = 192;
constexpr int kRouteJoinTokens = 2;
constexpr int kRouteDispatchSlots = 32;     // of those tokens, dispatched by the same CTA

inline RouteSplit route_split(int T_max, int E, int H, bool one_kernel = false)
{
    RouteSplit r;
    r.groups = (E + 15) / 16;
    const int eights = (T_max + 7) / 8;
    r.tiles = 1;
    while (r.tiles < 4 && r.tiles < eights && !(one_kernel && T_max <= 16) &&
           r.groups * ((eights + r.tiles - 1) / r.tiles) > 152 / 4)
        r.tiles *= 2;
    r.chunks = (eights + r.tiles - 1) / r.tiles;
    const int blocks = H / 64;
    const int want = 152 / (r.groups * r.chunks);
    r.slices = want < 1 ? 1 : (want < blocks ? want : blocks);
    r.join = T_max <= (one_kernel ? 16 : kRouteJoinTokens);   // tiles is 1 then
    return r;
}

// The tensor-core logits' tile (route_gemm.cu): experts of a tile and the CTAs
// of a cluster that share one 128-token tile's K.
struct RouteTile {
    int experts, slices;
};

// TMEM accumulators that a tile's K blocks go round
constexpr int route_accumulators(int experts) { return experts <= 128 ? 4 : 2; }

// The pair with the shortest estimate in cycles: waves of clusters over the
// GPU, each CTA its K blocks at their operand bytes at 64 a cycle (above the
// MMAs' cycles at these widths), the exchange of the partial rows and a fixed
// start and end. kHeld[s]: clusters of s one-per-SM CTAs that a GB300 holds at
// once, as its occupancy query reports; the 16 clusters of eight of T=1024,
// E=256, H=4096 run in two waves, 22.1 us against 14.3 in clusters of six.
// Measured otherwise (graph replays): T=2048, E=384, H=7168, 192 x 4 slices
// 22.5 us, 192 x 3 25.1, 256 x 4 24.1, 128 x 4 35.7; T=256, E=256, H=7168,
// 64 x 8 12.5, 128 x 8 14.3; T=8192, E=128, H=4096, 128 x 2 23.0, 64 x 1 30.2.
// Tiles whose chains of MMAs are longer than 80 are taken only if all are: the
// tensor cores truncate as they add (route_gemm.cu).
inline RouteTile route_tile(int T_max, int E, int H)
{
    constexpr int kHeld[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    RouteTile best = {64, 1};
    double best_cycles = 1e30;
    for (int n = 64; n <= 256; n += 64) {
        if (n > 64 && n - 64 >= E)
            break;
        for (int s = 1; s <= 8 && s <= H / 64; ++s) {
            const int blocks = (H / 64 + s - 1) / s;
            const int chain = 4 * ((blocks + route_accumulators(n) - 1) / route_accumulators(n));
            const long long clusters = ((static_cast<long long>(T_max) + 127) / 128) * ((E + n - 1) / n);
            const double waves = static_cast<double>((clusters + kHeld[s] - 1) / kHeld[s]);
            double cycles = waves * (3000.0 + blocks * 2.0 * (128 + n) + (s > 1 ? 128.0 * n * 4 / 32 : 0));
            if (chain > 80)
                cycles += 1e9 * chain;
            if (cycles < best_cycles) {
                best_cycles = cycles;
                best = {n, s};
            }
        }
    }
    return best;
}

// Floats of scratch: the slices' partial logits and sums of squares (few
// tokens), or the logits.
inline size_t route_scratch_floats(int T_max, int E, int H, bool normed)
{
    const size_t T = static_cast<size_t>(T_max);
    if (!normed && T_max > kRouteFewTokens)
        return T * E;
    return static_cast<size_t>(route_split(T_max, E, H).slices) * T * (E + 1);
}

// logits[t, e] for the rows t < T (T_max > kRouteFewTokens)
cudaError_t launch_route_gemm(const RouteArgs &a, float *logits, cudaStream_t stream, bool pdl);

cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream, bool pdl);

// ---- gradients (rows_backward.cu, expert_backward.cu, norm_backward.cu, route_backward.cu) ----

// dy_sorted[inv[t*k + j]] = bf16(w[t, j] * d_out[t]) and, with d_weights, the
// dot products <d_out[t], y_sorted[inv[t*k + j]]>
cudaError_t launch_combine_backward(const void *d_out, const float *y_sorted, const int32_t *inv,
                                    const float *topk_weights, const int32_t *d_num_tokens, int T_max, int k, int cap,
                                    int H, void *dy_sorted, float *d_weights, int num_sms, cudaStream_t stream);

// dx[t] = bf16(sum_j dx_sorted[inv[t*k + j]] + dx_add[t])
cudaError_t launch_dispatch_backward(const void *dx_sorted, bool f32, const int32_t *inv, const void *dx_add,
                                     const int32_t *d_num_tokens, int T_max, int k, int cap, int H, void *dx, int num_sms,
                                     cudaStream_t stream);

// act[r] = a and dgu[r] = [dg du] of the rows r < offsets[E], bf16, and row `cap` of both = 0 (expert_backward.cu)
cudaError_t launch_act_grad(const void *x, const void *dy, const void *W13, const void *W2, const int32_t *offsets,
                            int E, int cap, int H, int I, void *act, void *dgu, int32_t *err, int num_sms,
                            cudaStream_t stream);

// One grouped product of bf16 operands, for every expert e with the rows R_e =
// [offsets[e], offsets[e + 1]):
//  by_rows:  out[r, n] = sum_k a[r, k] b[e * b_expert_rows + k mod (64 wrap), n], r in R_e, k < 64 k_blocks
//  else:     out[e, m, n] = sum_{r in R_e} a[r, m] b[r, n], m < M
//  rows_on_n: out[e, n, m] = sum_{p < 2} sum_{r in R_e} a[r, m] b[r, n + p part_cols], m < M: as above with
//            the output transposed, for an N below 256 columns: the MMAs and B's loads follow it in steps of 128
// for n < N. a [a_rows, a_cols], b [b_rows, b_cols] and out ([cap, N], [E, M, N] or [E, N, M]) row-major.
struct ProductJob {
    int by_rows, rows_on_n;
    const void *a, *b;
    long long a_rows, a_cols, b_rows, b_cols;
    int M, N;
    int k_blocks, wrap, b_expert_rows;      // by_rows
    int part_cols;          // rows_on_n: from one part of b's columns to the next
    int zero_in_a;          // not by_rows: row `cap` of a (else of b) exists and holds zeros
    void *out;
    int out_f32;            // fp32, else bf16
    int accumulate;         // fp32, not by_rows: added to what is there
};

long long product_units(const ProductJob &j, int E, int cap);   // at most, for any offsets

// The ranges of rows: by offsets [E + 1], or E segments of segment_rows up to *num_rows (null: cap).
struct ProductRows {
    const int32_t *offsets;
    const int32_t *num_rows;
    int segment_rows;
};

// Up to three products in one launch; their rows are the same batch of `cap` rows. The
// kernel launched just before must let this one start only after a wait of its own for what
// came before it, and write neither offsets nor num_rows: they are read, and the units
// decoded, while it still runs.
cudaError_t launch_products(const ProductJob *jobs, int n, const ProductRows &rows, int E, int cap, int32_t *err,
                            int num_sms, cudaStream_t stream);

struct NormGradArgs {
    const void *h;             // bf16 or fp32
    const void *w;             // null: no weight
    const void *dx;            // bf16
    const void *dh_add;        // type of h; null: none
    const int32_t *d_num_tokens;
    void *dh;                  // type of h
    void *dw;                  // type of w; null: not wanted
    float *part;               // norm_grad_part_rows() x H partial sums of dw
    int32_t *err;
    int T_max, H;
    int h_f32, w_f32, unit_offset;
    float eps;
    long long h_stride, dx_stride, add_stride, out_stride;
};

int norm_grad_part_rows(int T_max, int H, bool h_f32);
cudaError_t launch_norm_backward(const NormGradArgs &a, cudaStream_t stream);

struct RouteGradArgs {
    const float *logits;       // [T_max, E]
    const int32_t *ids;        // [T_max, k]
    const float *d_weights;    // [T_max, k]
    const float *d_logits_add; // [T_max, E] or null
    const int32_t *d_num_tokens;
    float *d_logits;           // [T_max, E] or null
    void *parts;               // [T_max + 1, 2 Ep] bf16, Ep = E rounded up to 64: leading parts, then rests;
                               // the last row is set to zeros
    int32_t *err;
    int T_max, E, k;
    int sigmoid, renormalize;
    float scale;
};

cudaError_t launch_route_grad(const RouteGradArgs &a, int num_sms, cudaStream_t stream);

// The whole gradient where dl is zero but at the chosen experts and there are few
// slots, in all and of an expert on average. Graph replays, so and by the products:
// T=61, E=256, k=8, H=7168 9.6 us and 15.6; T=16, E=64, k=4, H=2048 2.7 and 7.8;
// T=128, E=384, k=8, H=7168 13.5 and 17.4; with 16 slots an expert (T=256, E=64,
// k=4, H=2048) 6.6 and 9.9, with 120 (T=120, E=8, k=8, H=4096) 13.3 and 9.5.
constexpr int kRouteFewSlots = 1024;

struct RouteFewArgs {
    const __nv_bfloat16 *x, *w;
    void *dx, *dw;             // null: not wanted
    int dw_f32, H;
};

inline bool route_grad_few(const RouteGradArgs &a)
{
    const long long slots = static_cast<long long>(a.T_max) * a.k;
    return !a.d_logits_add && (a.sigmoid || a.renormalize) && a.T_max <= 256 && slots <= kRouteFewSlots &&
           slots <= 16LL * a.E;
}

// (parts, offsets, segments of `a` are not used)
cudaError_t launch_route_grad_few(const RouteGradArgs &a, const RouteFewArgs &f, cudaStream_t stream);
// out[i] = sum_s part[s * n + i] in fp32, s ascending, stored as fp32 or bf16; n a multiple of 8
cudaError_t launch_sum_parts(const float *part, int parts, size_t n, void *out, bool f32, int num_sms,
                             cudaStream_t stream);

// 2-D bf16 tensor map [rows, cols] (cols contiguous), box of 64 columns x
// box_rows rows, 128-byte swizzle (grouped_gemm.cu).
bool make_tile_map(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint32_t box_rows);
// the same for fp32: boxes of 32 columns
bool make_tile_map_f32(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint32_t box_rows);

// number of SMs of the current device (cached)
int device_sm_count();

// host validation shared by the entry points (moe_api.cu)
moe_status_t validate_problem(const moe_problem_t *problem);
// (block_api.cu)
moe_status_t validate_norm(const moe_norm_problem_t *problem);
moe_status_t validate_router(const moe_router_problem_t *problem);
// rows of the sorted batch: the problem's capacity, or T_max * k when it is 0
int capacity_of(const moe_problem_t &problem);
// blocks of the multi-block dispatch: one per kDispatchSlotsPerBlock routed slots
long long dispatch_blocks(const moe_problem_t &problem);
moe_status_t validate_device();
// What moe_forward refuses beyond its pointers and workspace: a forward form
// or weight layout that the shape cannot take.
moe_status_t check_forward(const moe_problem_t &problem);
// The forward's problem when its rows are paired (moe_layer): twice the tokens,
// and a path of its own choice (an internal value; not for the entry points).
moe_problem_t paired_problem(const moe_problem_t &problem);
size_t forward_workspace_bytes(const moe_problem_t &problem);
// moe_forward after its checks. With `tail` (moe_layer) rows are paired: x has
// 2 T_max rows, the workspace is paired_problem's, and the combine's place is taken by
// launch_combine_residual, or by the end of the one-kernel form (`out` is then
// fp32 scratch [T_max, H], tail_sums tail_sum_floats of it), and the block's
// output goes into the residual stream as `tail` says. With `dispatched`, expert_offsets, perm
// and inv (forward_inv) are already written by the kernel before.
moe_status_t enqueue_forward(const moe_problem_t &problem, const void *x, const int32_t *topk_ids,
                             const float *topk_weights, const int32_t *d_num_tokens, const void *W13, const void *W2,
                             int32_t *expert_offsets, int32_t *perm, void *out, void *ws, cudaStream_t stream,
                             void *const *stage_events, const NormArgs *tail, bool dispatched,
                             float *tail_sums = nullptr);
int32_t *forward_inv(const moe_problem_t &problem, void *ws);
// bytes at the start of every workspace: the device error word and the
// counters that kernels leave at zero (moe_clear_device_error clears them)
size_t workspace_header_bytes();
// byte offset in that header of the router's counter
size_t route_counters_offset();
// whether launches for this problem use programmatic dependent launch (M-small path)
bool use_pdl(const moe_problem_t &problem);

}  // namespace moe
