/*
 * moe.h -- C ABI of libmoe.so: routed Mixture-of-Experts expert execution on
 * one NVIDIA GB300 (sm_103a), BF16 weights and activations, fp32 accumulation.
 *
 * The operation is the one the TileOps page "[Refactor][MoE] Separate
 * dispatched expert compute" (PR #1738) composes in its Summary: routed
 * expert execution = local dispatch -> dispatched-expert MLP compute on a
 * tight (no-pad) expert-major batch -> combine with the routing weights.
 * Its Scope fixes BF16 tight/no-pad expert compute and leaves the rows past
 * the valid-row count unspecified; its Summary keeps valid-row counts on the
 * GPU behind a static capacity so that a whole call replays under a CUDA
 * Graph.
 *
 * Notation: T tokens (T <= T_max), E experts, k experts per token, H hidden
 * size, I intermediate size, R = T*k routed slots, slot s = t*k + j,
 * cap = capacity (rows of the sorted batch, >= T_max*k).
 *
 * Conventions shared by every entry point:
 *  - Every pointer argument except `problem`, `bytes` and `host_code` is a
 *    DEVICE pointer on the current CUDA device, owned by the caller. The
 *    library never allocates or frees device memory and keeps no pointer
 *    after a call returns.
 *  - bf16 buffers are passed as `void*`: IEEE bfloat16, 2 bytes an element,
 *    row-major, rows contiguous. Every device buffer must be 16-byte aligned;
 *    the workspace 256-byte aligned.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream). Calls
 *    only enqueue work on it: they never synchronise the host, never read a
 *    device value on the host, and are legal inside CUDA stream capture
 *    (after the first call of the host thread on a device, which sets up
 *    function attributes; make that first call outside capture).
 *  - Several host threads may call at once, each with its own workspace and
 *    its own output buffers (on one stream or several): the library keeps
 *    its launch caches per host thread and all of a call's device state in
 *    its workspace.
 *  - Host validation fails closed: a status other than MOE_OK means nothing
 *    was enqueued (DeepGEMM page "MegaMoE: add cluster-paired FP4 weight
 *    packets", Scope and fallback: unsupported shapes fail closed during host
 *    validation). MOE_ERR_CUDA means a launch failed; the stream may then
 *    hold part of the call.
 *  - Problems seen on the device (an expert id outside [0, E) other than -1,
 *    a pipeline wait that gave up) never stop a call: they set bits in a
 *    sticky error word at the start of the workspace, read with
 *    moe_last_device_error().
 *  - The path of the expert GEMMs (large-tile or M-small weight streaming)
 *    is chosen on the host from the static shape only (TileOps page, Review
 *    follow-up: one effective grouped-GEMM kernel resolved up front, no
 *    runtime row-policy branch), never from device row counts.
 */
#ifndef MOE_GB300_MOE_H
#define MOE_GB300_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_NULL = 1,        /* a required pointer is NULL */
    MOE_ERR_SHAPE = 2,       /* a size is out of range or inconsistent */
    MOE_ERR_ALIGN = 3,       /* H or I not a multiple of 64 (of 128 for the PACKED and MXFP8 weight
                                layouts, moe_pack_weights and moe_quantize_weights), or a misaligned
                                buffer */
    MOE_ERR_WORKSPACE = 4,   /* ws_bytes smaller than moe_workspace_size() */
    MOE_ERR_UNSUPPORTED = 5, /* no GB300-class device, or a path this build lacks */
    MOE_ERR_CUDA = 6         /* a CUDA call failed */
} moe_status_t;

/* Bits of the device error word (moe_last_device_error). */
#define MOE_DEVERR_BAD_EXPERT_ID 0x1 /* an id outside [0, E) and not -1: slot dropped */
#define MOE_DEVERR_WAIT_TIMEOUT 0x2  /* a pipeline wait gave up: results of that call are invalid */
#define MOE_DEVERR_Y_RANGE 0x4       /* moe_forward, tiled paths: a down-GEMM output beyond the fp16
                                        range of its intermediate y was clipped to +-65504 */
#define MOE_DEVERR_BAD_LOGIT 0x8     /* moe_route, moe_layer: a router logit was NaN or +inf; that expert
                                        was not chosen for that token */

/* Expert-GEMM path. AUTO picks from the static shape, a = T_max*k/E routed
 * rows per expert on average: M-small for a <= 8, single-CTA tiles for
 * 8 < a < 128, CTA-pair tiles for a >= 128 (MXFP8 weights: M-small at
 * every a). */
typedef enum moe_path {
    MOE_PATH_AUTO = 0,
    MOE_PATH_TILED = 1,       /* 256-row activation tiles x 256-row weight tiles on CTA pairs (cta_group::2) */
    MOE_PATH_SMALL_M = 2,     /* weights on the MMA M side, token tiles of 16..64 rows */
    MOE_PATH_TILED_1CTA = 3   /* 128 x 256 tiles on single CTAs */
} moe_path_t;

typedef struct moe_problem {
    int32_t T_max;    /* maximum tokens of one call, >= 1 (static) */
    int32_t E;        /* experts, 1..1024 */
    int32_t k;        /* experts per token, 1..E */
    int32_t H;        /* hidden size, multiple of 64 (of 128 for PACKED and MXFP8 weights) */
    int32_t I;        /* intermediate size, multiple of 64 (of 128 for PACKED and MXFP8 weights) */
    int32_t capacity; /* rows of the sorted batch; 0 means T_max*k; else >= T_max*k */
    int32_t path;     /* moe_path_t */
    int32_t weight_layout; /* moe_weight_layout_t of W13 and W2 */
    int32_t forward_form;  /* moe_forward_form_t */
} moe_problem_t;

/* How moe_forward launches decode-size batches (M-small path, 16-row token
 * tiles). ONE_KERNEL: dispatch, both GEMMs and the combine as one persistent
 * kernel (results bit-identical to SEPARATE); moe_forward and
 * moe_resolve_profile return MOE_ERR_UNSUPPORTED for a problem that is not
 * decode-size or whose tables do not fit that kernel's shared memory.
 * SEPARATE: dispatch, the two fused GEMMs and the combine as three kernels
 * chained by programmatic dependent launch (for a few tokens with bf16
 * weights the GEMM kernel also dispatches the slots itself, with the same
 * result, so that it need not wait for the dispatch kernel). AUTO: SEPARATE (measured at one
 * token, E=384, H=7168, I=3072, down GEMM in 4 K parts: 129.6 vs 131.5 us
 * with bf16 weights, 117.3 vs 121.8 us with MXFP8 weights). Other problems
 * ignore the field. */
typedef enum moe_forward_form {
    MOE_FORWARD_AUTO = 0,
    MOE_FORWARD_SEPARATE = 1,
    MOE_FORWARD_ONE_KERNEL = 2
} moe_forward_form_t;

/* Layout of W13 / W2 in memory.
 *  ROW_MAJOR: W13[E, 2I, H], W2[E, H, I] bf16, row-major.
 *  PACKED: the output of moe_pack_weights. Same bytes, reordered in the order
 *  the GEMMs read them (DeepGEMM page "MegaMoE: add cluster-paired FP4 weight
 *  packets", Summary and Motivation: a weight layout that follows the kernel's
 *  access order, loaded through TMA descriptors): expert -> 128-row weight
 *  tile -> 64-wide K block, each block stored as the 128-byte-swizzled
 *  shared-memory image of its 128 rows x 64 columns (16 KB), the gate and up
 *  tiles of one W13 block side by side (32 KB). Every path reads it; results
 *  are bitwise identical to ROW_MAJOR. */
typedef enum moe_weight_layout {
    MOE_WEIGHTS_ROW_MAJOR = 0,
    MOE_WEIGHTS_PACKED = 1,
    MOE_WEIGHTS_MXFP8 = 2
} moe_weight_layout_t;

/* MXFP8: the pages' MXFP8 path with prequantized expert weights (FlashInfer
 * moe_ep page, PR #3980; format 32 e4m3 x e8m0), OCP Microscaling v1.0. Each
 * 32 consecutive elements of a row along K (H for W13, I for W2) share one
 * E8M0 scale X = 2^e; each element is an FP8 E4M3 code P; the weight is X * P.
 * The output of moe_quantize_weights, one buffer per matrix:
 *   codes:  [E, 2I, H] (W13) or [E, H, I] (W2) bytes, row-major;
 *   scales: right after the codes, rows*K/32 bytes in the order the decode
 *           GEMMs read them: for each 128-row tile (rows counted over all
 *           experts), each 128-wide K block: 128 rows x 4 bytes, the scales of
 *           the row's four 32-element sub-blocks; scale code = e + 127.
 * moe_forward reads MXFP8 weights on the M-small path, which MOE_PATH_AUTO
 * takes for this layout at every batch size (token tiles of 16, 32 or 64
 * rows by a = T_max*k/E): it streams the 1-byte codes and expands X * P to
 * bf16 on the chip, exactly, then multiplies by the bf16 activations as for
 * bf16 weights. Activations, h and the output stay bf16 (SiLU(gate)*up
 * rounded to bf16 as before), so the result is the bf16 forward on the
 * dequantized weights. Each token tile of an expert expands its weight tiles
 * again, so MXFP8 weights pay off up to about a = 32 (prefill at E=384: 17-19%
 * faster than bf16 weights) and cost time beyond: a = 64 18% slower, a = 128
 * 1.75x, a = 512 2.9x. A tiled path asked for explicitly and
 * moe_expert_compute return MOE_ERR_UNSUPPORTED for this layout. Weights must
 * be finite with every block maximum in [2^-110, 2^24). */

/* Bytes of workspace every entry point below needs for `problem` (pure host
 * arithmetic, no CUDA call). The same workspace serves all entry points; it
 * holds the device error word, the GEMM kernels' counters (readiness counts
 * and the GPU-wide counts their CTAs take units from), dispatch scratch, the
 * activation h[cap, I] and, for moe_forward, the sorted batches. A new
 * workspace must be zero-filled (cudaMemset, or moe_clear_device_error)
 * before its first moe_forward or moe_expert_compute call: with stale
 * counters the GEMMs would skip units. Every call leaves its counters at zero
 * again, also after a timed-out wait (FlashInfer moe_ep page, launch-path
 * notes: workspaces allocated zeroed, counters cleaned by the kernel's tail),
 * so no per-call clearing is needed. */
moe_status_t moe_workspace_size(const moe_problem_t *problem, size_t *bytes);

/* Which expert-GEMM path `problem` resolves to (MOE_PATH_TILED,
 * MOE_PATH_SMALL_M or MOE_PATH_TILED_1CTA) and its activation-tile height
 * per CTA. Pure host. */
moe_status_t moe_resolve_path(const moe_problem_t *problem, int32_t *path, int32_t *tile_rows);

/* The full static launch profile of `problem` on the current device: every
 * choice the library makes from shapes alone (FlashInfer moe_ep page: tile,
 * schedule and token-back knobs keyed on the compile-time maximum token
 * count). Queries the current device's SM count; enqueues nothing. */
typedef struct moe_profile {
    int32_t path;          /* moe_path_t that runs (never AUTO) */
    int32_t tile_rows;     /* activation rows of one CTA's tile */
    int32_t down_split_k;  /* 1, 2 or 4: K parts of the down GEMM, in separate fp32 buffers summed in part order */
    int32_t pdl;           /* 1: kernels of a call use programmatic dependent launch */
    int32_t fused_gather;  /* 1: moe_forward's gate-up GEMM gathers rows from x (no x_sorted) */
    int32_t cta_pair;      /* 1: tiled GEMMs run on 2-CTA clusters */
    int32_t fused_mlp;     /* 1: moe_forward runs both GEMMs as one persistent kernel */
    int32_t megakernel;    /* 1: moe_forward is that one kernel, dispatch and combine included */
    int32_t kernel_launches; /* kernels one moe_forward call launches (memsets not counted) */
} moe_profile_t;

moe_status_t moe_resolve_profile(const moe_problem_t *problem, moe_profile_t *profile);

/*
 * Local dispatch: routing -> tight expert-major batch (TileOps page,
 * Summary: local dispatch; Scope: tight/no-pad batch, valid rows read from
 * expert_offsets[-1:]).
 *   topk_ids[T_max, k] int32  expert of each slot; -1 = dropped slot.
 *   d_num_tokens       int32* device scalar T (<= T_max) read on the GPU, so
 *                      a captured graph can replay with a new token count;
 *                      NULL means T = T_max.
 *   expert_offsets[E+1] int32 out: exclusive prefix sum of the per-expert
 *                      slot counts; expert_offsets[E] = valid rows.
 *   perm[cap]   int32  out: perm[row] = slot, for row < expert_offsets[E]
 *                      (later rows unspecified). Inside one expert the rows
 *                      follow ascending slot order (stable scatter).
 *   inv[T_max*k] int32 out: inv[slot] = row, -1 for a dropped slot (slots of
 *                      tokens >= T are not written).
 *   x[T_max, H], x_sorted[cap, H] bf16: optional (both NULL or both set);
 *                      when set, x_sorted[row] = x[perm[row] / k].
 * Results are bit-exact and deterministic.
 */
moe_status_t moe_dispatch(const moe_problem_t *problem, const int32_t *topk_ids,
                          const int32_t *d_num_tokens, int32_t *expert_offsets,
                          int32_t *perm, int32_t *inv, const void *x, void *x_sorted,
                          void *ws, size_t ws_bytes, void *stream);

/*
 * Dispatched-expert MLP on the tight batch (TileOps page, Summary: expert
 * compute for tight expert-major batches; Review follow-up: fused-gated
 * epilogue). For every expert e and row r in [expert_offsets[e],
 * expert_offsets[e+1]):
 *   h[r, n]  = bf16( SiLU(sum_h x_sorted[r,h] W13[e,n,h]) * sum_h x_sorted[r,h] W13[e,I+n,h] )
 *   y_sorted[r, m] = sum_n h[r,n] W2[e,m,n]                       (fp32)
 * with fp32 accumulation on the tensor cores; h lives in the workspace.
 *   x_sorted[cap, H] bf16, W13[E, 2I, H] bf16 (rows 0..I-1 gate, I..2I-1 up),
 *   W2[E, H, I] bf16, y_sorted[cap, H] fp32 out (rows past the valid count
 *   are not written), expert_offsets[E+1] as produced by moe_dispatch.
 * y_sorted stays fp32 so that the combine rounds to bf16 once, at the end.
 * ws: a zero-filled workspace (see moe_workspace_size), left with its
 * counters at zero.
 */
moe_status_t moe_expert_compute(const moe_problem_t *problem, const void *x_sorted,
                                const int32_t *expert_offsets, const void *W13, const void *W2,
                                float *y_sorted, void *ws, size_t ws_bytes, void *stream);

/*
 * Combine (TileOps page, Summary: routing weights kept outside expert
 * compute): out[t, m] = bf16( sum_{j=0..k-1} w[t,j] * y_sorted[inv[t*k+j], m] ),
 * fp32, j ascending, dropped slots (inv = -1) skipped; deterministic.
 *   topk_weights[T_max, k] fp32, inv[T_max*k] int32, y_sorted[cap, H] fp32,
 *   out[T_max, H] bf16 (rows >= T untouched), d_num_tokens as above.
 */
moe_status_t moe_combine(const moe_problem_t *problem, const float *y_sorted, const int32_t *inv,
                         const float *topk_weights, const int32_t *d_num_tokens, void *out,
                         void *stream);

/*
 * The whole routed expert execution in one call: dispatch (with the row
 * gather) -> expert compute -> combine, all on `stream`, with the sorted
 * batches and inv held in the workspace. Arguments as above; perm and
 * expert_offsets are still returned to the caller. On the tiled paths
 * (prefill- and large-batch shapes) the intermediate y between the down GEMM
 * and the combine is kept in fp16 (round to nearest, saturating at +-65504:
 * a clipped value sets MOE_DEVERR_Y_RANGE), which halves its HBM traffic;
 * the separate moe_expert_compute / moe_combine keep y in fp32. Decode-size
 * batches keep y in fp32. For decode-size batches
 * (moe_profile_t.megakernel) the call is a single persistent kernel: every
 * CTA dispatches the call's slots itself, then runs its share of both GEMMs
 * and of the combine; its CTAs wait on one another (bounded), so it expects
 * the GPU's SMs free for its CTAs, one per SM, when it starts. Results equal
 * those of the separate entry points bit for bit.
 */
moe_status_t moe_forward(const moe_problem_t *problem, const void *x, const int32_t *topk_ids,
                         const float *topk_weights, const int32_t *d_num_tokens, const void *W13,
                         const void *W2, int32_t *expert_offsets, int32_t *perm, void *out,
                         void *ws, size_t ws_bytes, void *stream);

/*
 * moe_forward with stage timestamps: identical work, plus a cudaEventRecord of
 * stage_events[i] (cudaEvent_t, created by the caller with timing enabled)
 * at the 6 stage boundaries on `stream`: [0] before dispatch, [1] after the
 * dispatch kernels, [2] after the row gather, [3] after the gate-up GEMM,
 * [4] after the down GEMM, [5] after combine. Inside stream capture the
 * records become external event nodes of the graph (cudaEventRecordExternal),
 * so a replayed graph still reports per-stage times. No counterpart on the
 * pages: it exists to time each kernel from the host without a profiler.
 */
moe_status_t moe_forward_profiled(const moe_problem_t *problem, const void *x, const int32_t *topk_ids,
                                  const float *topk_weights, const int32_t *d_num_tokens, const void *W13,
                                  const void *W2, int32_t *expert_offsets, int32_t *perm, void *out,
                                  void *ws, size_t ws_bytes, void *stream, void *const *stage_events);

/*
 * moe_dispatch for callers that cannot allocate device memory. No counterpart
 * on the pages: some callers have no way to hand the library a workspace --
 * a runtime whose device memory is planned once at start-up and may not grow,
 * or code that runs under stream capture, where cudaMalloc is not allowed.
 * This variant takes no workspace: its per-block counts live in a static
 * device array of MOE_NOALLOC_SCRATCH_INTS int32 (1 MiB) inside libmoe.so,
 * which every GPU that loads the library keeps until the process exits.
 * Inputs and outputs are the caller's, exactly as in moe_dispatch, and the
 * results are identical to moe_dispatch's. Differences:
 *  - Returns MOE_ERR_WORKSPACE, before touching the device, when the problem
 *    needs more than the static array: 64 + 2 * ceil(T_max*k / 1024) * E ints.
 *  - The first call on a device looks up the array's device address with
 *    that device current, and looks it up again when the device's current
 *    context has changed since (cudaDeviceReset, a new primary context);
 *    make the first call in each context before any stream capture.
 *  - All calls share the one array, which keeps the previous call's contents
 *    (each call rewrites what it reads). Calls that overlap on the GPU --
 *    different streams without ordering between them -- race on it: order
 *    them on one stream.
 *  - An invalid expert id is dropped as in moe_dispatch, but its error bit
 *    goes to the static array and is not reported.
 * It allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 */
#define MOE_NOALLOC_SCRATCH_INTS 262144
moe_status_t moe_dispatch_noalloc(const moe_problem_t *problem, const int32_t *topk_ids,
                                  const int32_t *d_num_tokens, int32_t *expert_offsets,
                                  int32_t *perm, int32_t *inv, const void *x, void *x_sorted,
                                  void *stream);

/*
 * Reorder W13 and W2 (row-major) into the PACKED layout, once, at model load.
 * W13_packed and W2_packed have the sizes of W13 and W2 and must not overlap
 * them. Only problem->E, H and I matter. Enqueued on `stream`.
 */
moe_status_t moe_pack_weights(const moe_problem_t *problem, const void *W13, const void *W2, void *W13_packed,
                              void *W2_packed, void *stream);

/* Bytes of W13 and W2 in `layout` (ROW_MAJOR and PACKED: 2 per element;
 * MXFP8: 1 per element plus one scale byte per 32). Pure host. */
moe_status_t moe_weight_bytes(const moe_problem_t *problem, int32_t layout, size_t *w13_bytes,
                              size_t *w2_bytes);

/* Quantize W13 and W2 (row-major bf16) to the MXFP8 layout, once, at model
 * load. W13_mx and W2_mx have moe_weight_bytes(MXFP8) bytes and must not
 * overlap the sources. Only problem->E, H and I matter. Enqueued on `stream`.
 * Bit-exact with the OCP MX definition above (round to nearest even,
 * saturation at 448). */
moe_status_t moe_quantize_weights(const moe_problem_t *problem, const void *W13, const void *W2,
                                  void *W13_mx, void *W2_mx, void *stream);

/* ------------------------------------------------------------------------
 * The block around the expert execution: the norm of the residual stream
 * before it, the router, and the way back into the residual stream (norm,
 * gate, residual scale), each as its own entry point and, for a few tokens,
 * together with the experts as one call (moe_layer). The conventions above
 * hold: device pointers, 16-byte alignment, no allocation, no host
 * synchronisation, legal inside stream capture, statuses fail closed. An
 * operator reads and writes the rows t < T only (T as d_num_tokens gives it,
 * T_max when that is NULL). The pages leave the router and the norms outside
 * the path (TileOps page, Summary: routing weights kept outside expert
 * compute); the formulas below are the usual ones of such models.
 * ------------------------------------------------------------------------ */

typedef enum moe_dtype {
    MOE_DTYPE_BF16 = 0,
    MOE_DTYPE_FP32 = 1
} moe_dtype_t;

/* The gate g of moe_norm_residual and moe_layer. */
typedef enum moe_gate {
    MOE_GATE_NONE = 0,     /* 1 */
    MOE_GATE_CHANNEL = 1,  /* g[H], w_dtype: one value per channel (a learned layer scale) */
    MOE_GATE_TOKEN = 2,    /* g[T_max] fp32: one value per token */
    MOE_GATE_ELEMENT = 3   /* g[T_max, H] bf16, rows gate_stride apart */
} moe_gate_t;

typedef struct moe_norm_problem {
    int32_t T_max;          /* maximum tokens, 1..2^30 */
    int32_t H;              /* hidden size, a multiple of 64, at most 32768 */
    int32_t h_dtype;        /* moe_dtype_t of the residual stream (h and h_out) */
    int32_t w_dtype;        /* moe_dtype_t of the norm weights and of the channel gate */
    int32_t unit_offset;    /* 1: a norm multiplies by 1 + w instead of w */
    int32_t norm_block;     /* moe_norm_residual, moe_layer: 1: y is normalised, 0: taken as it is */
    int32_t gate;           /* moe_gate_t */
    float eps;              /* > 0, finite */
    float residual_scale;   /* s, finite */
    int64_t h_stride;       /* elements between rows: 0 means H; else >= H and a multiple of 8 */
    int64_t y_stride;
    int64_t x_stride;       /* of x (moe_norm) and x_next */
    int64_t out_stride;     /* of h_out */
    int64_t gate_stride;    /* of an ELEMENT gate */
} moe_norm_problem_t;

/*
 * Norm before the block: x[t, m] = bf16( h[t, m] * r_t * w[m] ),
 * r_t = 1 / sqrt( mean_m h[t, m]^2 + eps ), in fp32 with one rounding.
 *   h[T_max, H] of h_dtype, w[H] of w_dtype or NULL (no weight),
 *   x[T_max, H] bf16 out; x must not overlap h.
 * norm_block, gate and residual_scale are not read.
 */
moe_status_t moe_norm(const moe_norm_problem_t *problem, const void *h, const void *w, const int32_t *d_num_tokens,
                      void *x, void *stream);

/*
 * Back into the residual stream, and the next norm in the same pass:
 *   n[t, m]      = y[t, m] * r(y_t) * w_post[m]      (norm_block; else y[t, m])
 *   h_out[t, m]  = h[t, m] + s * g * n[t, m]
 *   x_next[t, m] = bf16( h'[t, m] * r(h'_t) * w_next[m] ), h' = h_out before its rounding
 * in fp32, one rounding per output.
 *   y[T_max, H] bf16 (moe_forward's out), gate as `gate` says (NULL for
 *   MOE_GATE_NONE), w_post and w_next [H] or NULL (no weight), h_out of
 *   h_dtype, x_next bf16 or NULL (not computed). h_out may be h itself, with
 *   the same stride; no other buffers may overlap.
 */
moe_status_t moe_norm_residual(const moe_norm_problem_t *problem, const void *h, const void *y, const void *w_post,
                               const void *gate, const void *w_next, const int32_t *d_num_tokens, void *h_out,
                               void *x_next, void *stream);

/* Score of an expert from its logit. */
typedef enum moe_score {
    MOE_SCORE_SOFTMAX = 0,  /* softmax over all E experts */
    MOE_SCORE_SIGMOID = 1
} moe_score_t;

typedef struct moe_router_problem {
    int32_t T_max;        /* maximum tokens, >= 1 */
    int32_t E;            /* experts, 1..1024 */
    int32_t k;            /* experts per token, 1..64, at most topk_group * E / n_group */
    int32_t H;            /* hidden size, multiple of 64 */
    int32_t score;        /* moe_score_t */
    int32_t renormalize;  /* 1: a token's k scores are divided by their sum */
    int32_t n_group;      /* groups of consecutive experts, 1..32, dividing E; 1: no groups */
    int32_t topk_group;   /* groups kept per token, 1..n_group */
    int32_t group_top;    /* a group's value is the sum of its 1 or 2 largest keys */
    float scale;          /* the weights are multiplied by it; finite */
} moe_router_problem_t;

/* Bytes of workspace of moe_route (pure host). Zero-filled before its first
 * use, like every workspace; holds the device error word at its start. */
moe_status_t moe_route_workspace_size(const moe_router_problem_t *problem, size_t *bytes);

/*
 * Router: logits[t, e] = sum_m x[t, m] w_router[e, m] in fp32, the score of
 * each expert, and the k experts of the largest keys.
 *  - key = score + bias; without a bias and with group_top = 1 the logit
 *    itself (the same order, with no ties from rounding the score);
 *  - n_group > 1: only the topk_group groups of the largest value keep their
 *    experts (ties to the lower group);
 *  - ids in descending key order, ties to the lower expert;
 *  - weight = scale * score (without the bias), divided by the sum of the
 *    chosen scores when renormalize is set.
 * An expert whose key is -inf or NaN is never chosen: a bias of -inf switches
 * an expert off. A token with fewer than k such experts gets id -1 (a dropped
 * slot for moe_dispatch) and weight 0 in the remaining places. A logit that
 * is NaN or +inf sets MOE_DEVERR_BAD_LOGIT and is taken as -inf.
 *   x[T_max, H] bf16, w_router[E, H] bf16, bias[E] fp32 or NULL,
 *   topk_ids[T_max, k] int32 and topk_weights[T_max, k] fp32 out,
 *   logits[T_max, E] fp32 out or NULL.
 * Deterministic. ws as moe_route_workspace_size says; the calls that share
 * one workspace are ordered on one stream.
 */
moe_status_t moe_route(const moe_router_problem_t *problem, const void *x, const void *w_router, const float *bias,
                       const int32_t *d_num_tokens, int32_t *topk_ids, float *topk_weights, float *logits, void *ws,
                       size_t ws_bytes, void *stream);

#define MOE_LAYER_MAX_TOKENS 128

/* The three parts agree in T_max (at most MOE_LAYER_MAX_TOKENS), H, E and k;
 * H is at most 16384. The layer's sorted rows are its own and follow T_max * k:
 * a larger experts.capacity changes nothing. */
typedef struct moe_layer_problem {
    moe_problem_t experts;
    moe_router_problem_t router;
    moe_norm_problem_t norm;
} moe_layer_problem_t;

moe_status_t moe_layer_workspace_size(const moe_layer_problem_t *problem, size_t *bytes);

/*
 * The whole block for a few tokens (a decode step):
 *   v = h * r(h) * w_pre            the norm, unrounded
 *   ids, weights = the router on v  (as moe_route, but on v before its rounding)
 *   y = the experts on v, weighted and summed, unrounded
 *   h_out, x_next                   as moe_norm_residual, from y before its rounding
 * The experts' matrix instructions take bf16 activations; v and the experts'
 * inner activations go to them as two bf16 rows each, leading part and rest,
 * so they count with 16 bits, not 24 (a few tokens leave the token tiles mostly
 * empty, so the second row costs nothing to speak of). Against 64 bits y is off by
 * 5e-6 of its rms at H=1024, I=512 and 1.7e-5 at H=7168, I=2048, where the tensor
 * cores' truncating sums add theirs; in 32 bits throughout it would be 1e-6 and
 * 4e-7. A bf16 stream's own rounding hides that (1 of 200 elements of h_out
 * rounds to the other neighbour); an fp32 stream carries it. experts.path AUTO
 * picks the token tiles for paired rows (16 or 32 rows, or the tiled path's
 * 128); MOE_PATH_TILED runs as MOE_PATH_TILED_1CTA. With experts.forward_form MOE_FORWARD_ONE_KERNEL the
 * call is two kernels for up to 16 tokens (three beyond): norm and router,
 * then all the rest; as in moe_forward its CTAs wait on one another and the
 * form is refused for problems it does not fit (MXFP8 weights with more than
 * two paired rows an expert on average among them). Otherwise: norm and router,
 * one kernel for T_max <= 2, two beyond; the dispatch, inside that kernel for
 * T_max <= 2 with T_max*k <= 32, else one kernel (three above 1024 slots); a
 * gather of the rows for MXFP8 weights and for 128-row tiles; the experts, one
 * kernel with 16-row tiles or MXFP8 weights, else two; combine and residual. So
 * a decoded token takes three kernels with bf16 weights and four with MXFP8. The
 * call beats its four pieces up to about 64 tokens; at 128 the pieces, whose
 * experts read bf16 x, took 4% to 12% less. Arguments as in moe_norm,
 * moe_route, moe_forward and moe_norm_residual; w_pre, w_post and w_next
 * follow norm.w_dtype. topk_ids, topk_weights,
 * expert_offsets and perm are outputs. More tokens than MOE_LAYER_MAX_TOKENS
 * return MOE_ERR_SHAPE: call moe_norm, moe_route, moe_forward and
 * moe_norm_residual in turn (there the router and the experts read the
 * rounded x). h_out may be h; no other buffers may overlap.
 */
moe_status_t moe_layer(const moe_layer_problem_t *problem, const void *h, const void *w_pre, const void *w_router,
                       const float *bias, const void *W13, const void *W2, const void *w_post, const void *gate,
                       const void *w_next, const int32_t *d_num_tokens, int32_t *topk_ids, float *topk_weights,
                       int32_t *expert_offsets, int32_t *perm, void *h_out, void *x_next, void *ws, size_t ws_bytes,
                       void *stream);

/* ------------------------------------------------------------------------
 * Training: the gradients of the operators above. Written g for "gradient of
 * the loss by": d_out = g(out) and so on. The conventions above hold. Nothing
 * is kept from the forward calls but what the arguments name: the routing's
 * maps (inv and expert_offsets of moe_dispatch), the sorted rows x_sorted, the
 * experts' y_sorted (only if the routing weights' gradient is wanted) and the
 * router's logits. The chain of one block, last to first:
 *   moe_combine_backward   d_out           -> dy_sorted, d_weights
 *   moe_expert_backward    dy_sorted       -> dx_sorted, dW13, dW2
 *   moe_route_backward     d_weights       -> dx (the router's part), dw_router
 *   moe_dispatch_backward  dx_sorted       -> dx (all of it)
 *   moe_norm_backward      dx              -> dh, dw
 * Every operator is deterministic: sums go in a fixed order, no atomics. Buffers
 * do not overlap but where an entry point says so.
 * ------------------------------------------------------------------------ */

/*
 * Gradient of moe_combine, for r = inv[t*k + j]:
 *   dy_sorted[r, m]  = bf16( w[t, j] * d_out[t, m] )
 *   d_weights[t, j]  = sum_m d_out[t, m] y_sorted[r, m]       (fp32)
 *   d_out[T_max, H] bf16, y_sorted[cap, H] fp32 (NULL without d_weights),
 *   inv[T_max*k] and topk_weights[T_max, k] as for moe_combine (no two slots
 *   with one row; a row outside [0, cap) counts as dropped),
 *   dy_sorted[cap, H] bf16 out: rows that no slot holds are not written,
 *   d_weights[T_max, k] fp32 out, 0 for a dropped slot, or NULL (not wanted).
 * Slots of tokens >= T are not read or written.
 */
moe_status_t moe_combine_backward(const moe_problem_t *problem, const void *d_out, const float *y_sorted,
                                  const int32_t *inv, const float *topk_weights, const int32_t *d_num_tokens,
                                  void *dy_sorted, float *d_weights, void *stream);

/*
 * Gradient of moe_dispatch's row gather:
 *   dx[t, m] = bf16( sum_{j = 0..k-1} dx_sorted[inv[t*k + j], m] + dx_add[t, m] )
 * in fp32, j ascending, dropped slots skipped, dx_add last.
 *   dx_sorted[cap, H] of dx_dtype (moe_dtype_t), dx_add[T_max, H] bf16 or NULL
 *   (the gradient that reaches x on another path, the router's), dx[T_max, H]
 *   bf16 out, rows >= T untouched. dx may be dx_add; inv as above.
 */
moe_status_t moe_dispatch_backward(const moe_problem_t *problem, int32_t dx_dtype, const void *dx_sorted,
                                   const int32_t *inv, const void *dx_add, const int32_t *d_num_tokens, void *dx,
                                   void *stream);

typedef struct moe_expert_grad_problem {
    moe_problem_t experts;  /* weight_layout ROW_MAJOR (others: MOE_ERR_UNSUPPORTED); path and forward_form are not read */
    int32_t dx_dtype;       /* moe_dtype_t of dx_sorted */
    int32_t dw_dtype;       /* moe_dtype_t of dW13 and dW2 */
    int32_t accumulate;     /* 1: the weight gradients are added to what dW13 and dW2 hold (FP32 only) */
} moe_expert_grad_problem_t;

/* Bytes of workspace of moe_expert_backward: the device error word and 6 bytes
 * for each of cap * I elements (pure host). Zero-filled before its first use. */
moe_status_t moe_expert_backward_workspace_size(const moe_expert_grad_problem_t *problem, size_t *bytes);

/*
 * Gradient of moe_expert_compute. With g, u the gate and up products of the
 * rows (computed again), s = 1 / (1 + exp(-g)), a = g s u, of each expert e and
 * its rows r:
 *   da[r]  = dy_sorted[r] W2[e],  du = da g s,  dg = da u s (1 + g (1 - s))
 *   dx_sorted[r] = [dg du][r] W13[e]
 *   dW2[e]  = sum_r dy_sorted[r]^T a[r],  dW13[e] = sum_r [dg du][r]^T x_sorted[r]
 * fp32 sums on the tensor cores, whose additions truncate (a sum of n products is
 * off by up to (n / 16 + 32) 2^-23 of the sum of their |values|: n rows of an expert
 * for its weight gradients); a and [dg du] are rounded to bf16 once, as
 * their operands, and each output once. An expert without rows gets zero
 * weight gradients (none added with `accumulate`).
 *   x_sorted, dy_sorted [cap, H] bf16; expert_offsets[E+1] of moe_dispatch (or
 *   any non-decreasing offsets, clamped to [0, cap]); W13, W2 as for
 *   moe_expert_compute; dx_sorted[cap, H], dW13[E, 2I, H], dW2[E, H, I] out, each
 *   NULL if not wanted, not all. Rows of dx_sorted at and past
 *   expert_offsets[E] are not written; rows of the inputs there do not count,
 *   whatever they hold. A row that is not finite leaves its own expert's weight
 *   gradients not finite (an infinity may come out as NaN), no other's.
 */
moe_status_t moe_expert_backward(const moe_expert_grad_problem_t *problem, const void *x_sorted,
                                 const int32_t *expert_offsets, const void *W13, const void *W2, const void *dy_sorted,
                                 void *dx_sorted, void *dW13, void *dW2, void *ws, size_t ws_bytes, void *stream);

/* Bytes of workspace of moe_norm_backward (pure host). */
moe_status_t moe_norm_backward_workspace_size(const moe_norm_problem_t *problem, size_t *bytes);

/*
 * Gradient of moe_norm (and, with dh_add, of moe_norm_residual's next norm),
 * r_t and the weight w' (w, or 1 + w with unit_offset) as there, q = dx * w':
 *   dh[t, m] = r_t ( q[t, m] - h[t, m] r_t^2 mean_m(q h) ) + dh_add[t, m]
 *   dw[m]    = sum_{t < T} dx[t, m] h[t, m] r_t
 * in fp32, one rounding per output.
 *   h[T_max, H] of h_dtype, rows h_stride apart; w[H] of w_dtype or NULL (no
 *   weight); dx[T_max, H] bf16, rows x_stride apart; dh_add[T_max, H] of
 *   h_dtype, rows y_stride apart, or NULL (the gradient that reaches h past the
 *   block); dh[T_max, H] of h_dtype out, rows out_stride apart; dw[H] of
 *   w_dtype out, or NULL. dh may be h or dh_add, with the same stride; no other
 *   buffers may overlap.
 * norm_block, gate and residual_scale are not read. ws: only its device error
 * word has to start at zero (a wait inside the kernel that gave up sets
 * MOE_DEVERR_WAIT_TIMEOUT).
 */
moe_status_t moe_norm_backward(const moe_norm_problem_t *problem, const void *h, const void *w, const void *dx,
                               const void *dh_add, const int32_t *d_num_tokens, void *dh, void *dw, void *ws,
                               size_t ws_bytes, void *stream);

/* Bytes of workspace of moe_route_backward (pure host). Zero-filled before its
 * first use; holds the device error word at its start. */
moe_status_t moe_route_backward_workspace_size(const moe_router_problem_t *problem, size_t *bytes);

/*
 * Gradient of moe_route by its weights:
 *   d_logits[t, e] = g(logits) from d_weights through the score, renormalising
 *                    and scale, plus d_logits_add[t, e]              (fp32)
 *   dx[t, m]       = bf16( sum_e d_logits[t, e] w_router[e, m] )
 *   dw_router[e,m] = sum_{t < T} d_logits[t, e] x[t, m]
 * The choice of experts and the selection bias have no gradient. The products
 * take d_logits with 16 bits (two bf16 parts; a relative 2^-16) and sum in fp32
 * on the tensor cores, whose additions truncate: dx is off by up to (E / 8 + 32) 2^-23
 * of the sum of its |terms|, dw_router by up to 6.5e-5 of its own, since no such sum
 * goes over more than 4096 tokens (T / 1024 past 4 million): those of the ranges
 * are added in fp32, 2^-24 each.
 * Logits that are NaN or +inf count as -inf, whose gradient is 0; an id of -1
 * adds nothing, an id outside [0, E) neither and sets MOE_DEVERR_BAD_EXPERT_ID.
 *   x[T_max, H] bf16 (NULL without dw_router), w_router[E, H] bf16 (NULL without
 *   dx), logits[T_max, E], topk_ids[T_max, k] as moe_route wrote them,
 *   d_weights[T_max, k] fp32, d_logits_add[T_max, E] fp32 or NULL (an auxiliary
 *   loss's gradient); dx, dw_router[E, H] of dw_dtype (moe_dtype_t) and
 *   d_logits[T_max, E] fp32 out, each NULL if not wanted, not all. Rows >= T of
 *   dx and d_logits are not written. d_logits may be d_logits_add.
 */
moe_status_t moe_route_backward(const moe_router_problem_t *problem, int32_t dw_dtype, const void *x,
                                const void *w_router, const float *logits, const int32_t *topk_ids,
                                const float *d_weights, const float *d_logits_add, const int32_t *d_num_tokens,
                                void *dx, void *dw_router, float *d_logits, void *ws, size_t ws_bytes, void *stream);

/* Read the sticky device error word of `ws` into *host_code (0 = none).
 * Synchronises `stream` (the only entry point that does). */
moe_status_t moe_last_device_error(const void *ws, void *stream, int32_t *host_code);

/* Clear the device error word and the GEMM kernels' counters (enqueued on
 * `stream`); also readies a workspace of unknown contents for moe_forward
 * and moe_expert_compute. */
moe_status_t moe_clear_device_error(void *ws, void *stream);

/* Human-readable name of a status. Never NULL. */
const char *moe_status_string(moe_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_MOE_H */
