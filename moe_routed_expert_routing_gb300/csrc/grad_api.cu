// grad_api.cu -- C ABI of the block's gradients (declared and documented in
// include/moe.h). Host side only: validation (fails closed before any
// launch), workspace layout and launches.
#include <cmath>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool is_dtype(int32_t d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_FP32; }

template <typename T>
T *at(void *ws, size_t off)
{
    return reinterpret_cast<T *>(static_cast<uint8_t *>(ws) + off);
}

moe_status_t check_ws(const void *ws, size_t have, size_t need)
{
    if (!ws)
        return MOE_ERR_NULL;
    if (!aligned(ws, 256))
        return MOE_ERR_ALIGN;
    return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

// ---- experts ----

// Workspace: the header (error word), a [cap + 1, I] and [dg du] [cap + 1, 2I] in bf16.
struct ExpertLayout {
    size_t act, dgu, total;
};

ExpertLayout expert_layout(const moe_problem_t &p)
{
    const size_t cap = static_cast<size_t>(capacity_of(p)), I = static_cast<size_t>(p.I);
    ExpertLayout L;
    L.act = workspace_header_bytes();
    L.dgu = align_up(L.act + 2 * (cap + 1) * I);
    L.total = align_up(L.dgu + 4 * (cap + 1) * I);
    return L;
}

moe_status_t check_expert_grad(const moe_expert_grad_problem_t *p)
{
    if (!p)
        return MOE_ERR_NULL;
    const moe_status_t st = validate_problem(&p->experts);
    if (st != MOE_OK)
        return st;
    if (!is_dtype(p->dx_dtype) || !is_dtype(p->dw_dtype) || (p->accumulate != 0 && p->accumulate != 1) ||
        (p->accumulate && p->dw_dtype != MOE_DTYPE_FP32))
        return MOE_ERR_SHAPE;
    if (p->experts.weight_layout != MOE_WEIGHTS_ROW_MAJOR)
        return MOE_ERR_UNSUPPORTED;
    // units of the products are counted in 32 bits
    const long long cap = capacity_of(p->experts), E = p->experts.E, H = p->experts.H, I = p->experts.I;
    const long long nh = (H + 255) / 256, ni = (I + 255) / 256, n2i = (2 * I + 255) / 256;
    const long long tiles = (cap + 255) / 256 + E;
    if (tiles * nh + E * nh * ni + E * n2i * nh > (1LL << 31) - 1 || tiles * ((I + 127) / 128) > (1LL << 31) - 1)
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

// ---- norm ----

struct NormGradLayout {
    size_t part, total;
};

NormGradLayout norm_layout(const moe_norm_problem_t &p)
{
    NormGradLayout L;
    L.part = workspace_header_bytes();
    L.total = align_up(L.part + sizeof(float) * static_cast<size_t>(p.H) *
                                    norm_grad_part_rows(p.T_max, p.H, p.h_dtype == MOE_DTYPE_FP32));
    return L;
}

// ---- router ----

// Token ranges whose products for dw_router are summed apart, so that a
// [E, H] result with few tiles still fills the GPU: a unit for each of a
// GB300's 76 CTA pairs, or two where that leaves one range. A range is one
// unbroken sum on the tensor cores, whose additions truncate: (2 rows / 16) of them, 2^-23 of
// the sum each at most, so ranges have kRangeRows tokens at most and their sums are
// added in fp32. Same-signed terms with T=262144, E=128, H=4096 were off by 4.5e-4 of
// dw in four ranges, and by 1.7e-5 in 64. The call's time at T=65536 with E=128, H=4096
// 255 us in four ranges, 269 in 16, with E=384, H=7168 1044 in two and 975 in 16; T=8192,
// E=1024, H=7168 289 in one and 306 in two. (More than kRangeRows * kMaxExperts
// tokens, 4.2 million, go in kMaxExperts longer ranges.)
constexpr int kRangeRows = 4096;

struct RouteSplitK {
    int segments, rows;
};

RouteSplitK route_segments(const moe_router_problem_t &p)
{
    const long long tiles = ((p.E + 255LL) / 256) * ((p.H + 255LL) / 256);
    long long want = 76 / tiles;
    if (want < 2)
        want = 152 / tiles;
    if (want < 1)
        want = 1;
    const long long fill = (p.T_max + want - 1) / want, least = (p.T_max + kMaxExperts - 1LL) / kMaxExperts;
    long long rows = fill < kRangeRows ? fill : kRangeRows;
    rows = ((rows > least ? rows : least) + 255) / 256 * 256;
    return {static_cast<int>((p.T_max + rows - 1) / rows), static_cast<int>(rows)};
}

struct RouteGradLayout {
    size_t parts, sums, total;
};

moe_status_t check_route_grad(const moe_router_problem_t *p)
{
    const moe_status_t st = validate_router(p);
    if (st != MOE_OK)
        return st;
    // units of the products are counted in 32 bits
    const RouteSplitK s = route_segments(*p);
    const long long nh = (p->H + 255LL) / 256, ne = (p->E + 127LL) / 128;
    if (((p->T_max + 255LL) / 256 + s.segments + s.segments * ne) * nh > (1LL << 31) - 1)
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

RouteGradLayout route_grad_layout(const moe_router_problem_t &p)
{
    const RouteSplitK s = route_segments(p);
    const size_t Ep = (p.E + 63) / 64 * 64;
    RouteGradLayout L;
    L.parts = align_up(workspace_header_bytes());
    L.sums = align_up(L.parts + 4 * Ep * (static_cast<size_t>(p.T_max) + 1));
    const size_t sums = s.segments > 1 ? sizeof(float) * s.segments * p.E * static_cast<size_t>(p.H) : 0;
    L.total = align_up(L.sums + sums);
    return L;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_combine_backward(const moe_problem_t *problem, const void *d_out, const float *y_sorted,
                                  const int32_t *inv, const float *topk_weights, const int32_t *d_num_tokens,
                                  void *dy_sorted, float *d_weights, void *stream)
{
    moe_status_t st = validate_problem(problem);
    if (st != MOE_OK)
        return st;
    if (!d_out || !inv || !topk_weights || !dy_sorted || (d_weights && !y_sorted))
        return MOE_ERR_NULL;
    for (const void *q : {d_out, static_cast<const void *>(y_sorted), static_cast<const void *>(dy_sorted)})
        if (!aligned(q, 16))
            return MOE_ERR_ALIGN;
    if ((st = validate_device()) != MOE_OK)
        return st;
    const moe_problem_t &p = *problem;
    return cuda_status(launch_combine_backward(d_out, y_sorted, inv, topk_weights, d_num_tokens, p.T_max, p.k,
                                               capacity_of(p), p.H, dy_sorted, d_weights, device_sm_count(),
                                               static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_dispatch_backward(const moe_problem_t *problem, int32_t dx_dtype, const void *dx_sorted,
                                   const int32_t *inv, const void *dx_add, const int32_t *d_num_tokens, void *dx,
                                   void *stream)
{
    moe_status_t st = validate_problem(problem);
    if (st != MOE_OK)
        return st;
    if (!is_dtype(dx_dtype))
        return MOE_ERR_SHAPE;
    if (!dx_sorted || !inv || !dx)
        return MOE_ERR_NULL;
    for (const void *q : {dx_sorted, dx_add, static_cast<const void *>(dx)})
        if (!aligned(q, 16))
            return MOE_ERR_ALIGN;
    if ((st = validate_device()) != MOE_OK)
        return st;
    const moe_problem_t &p = *problem;
    return cuda_status(launch_dispatch_backward(dx_sorted, dx_dtype == MOE_DTYPE_FP32, inv, dx_add, d_num_tokens,
                                                p.T_max, p.k, capacity_of(p), p.H, dx, device_sm_count(),
                                                static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_backward_workspace_size(const moe_expert_grad_problem_t *problem, size_t *bytes)
{
    if (!bytes)
        return MOE_ERR_NULL;
    const moe_status_t st = check_expert_grad(problem);
    if (st != MOE_OK)
        return st;
    *bytes = expert_layout(problem->experts).total;
    return MOE_OK;
}

moe_status_t moe_expert_backward(const moe_expert_grad_problem_t *problem, const void *x_sorted,
                                 const int32_t *expert_offsets, const void *W13, const void *W2, const void *dy_sorted,
                                 void *dx_sorted, void *dW13, void *dW2, void *ws, size_t ws_bytes, void *stream)
{
    moe_status_t st = check_expert_grad(problem);
    if (st != MOE_OK)
        return st;
    if (!x_sorted || !expert_offsets || !W13 || !W2 || !dy_sorted || (!dx_sorted && !dW13 && !dW2))
        return MOE_ERR_NULL;
    for (const void *q : {x_sorted, W13, W2, dy_sorted, static_cast<const void *>(dx_sorted),
                          static_cast<const void *>(dW13), static_cast<const void *>(dW2)})
        if (!aligned(q, 16))
            return MOE_ERR_ALIGN;
    const moe_problem_t &p = problem->experts;
    const ExpertLayout L = expert_layout(p);
    if ((st = check_ws(ws, ws_bytes, L.total)) != MOE_OK || (st = validate_device()) != MOE_OK)
        return st;
    const int sms = device_sm_count(), cap = capacity_of(p);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void *act = at<void>(ws, L.act), *dgu = at<void>(ws, L.dgu);
    int32_t *err = at<int32_t>(ws, 0);
    if ((st = cuda_status(launch_act_grad(x_sorted, dy_sorted, W13, W2, expert_offsets, p.E, cap, p.H, p.I, act, dgu,
                                          err, sms, s))) != MOE_OK)
        return st;
    ProductJob jobs[3];
    int n = 0;
    if (dx_sorted) {
        ProductJob j = {};
        j.by_rows = 1;
        j.a = dgu;
        j.a_rows = cap;
        j.a_cols = 2LL * p.I;
        j.b = W13;
        j.b_rows = 2LL * p.I * p.E;
        j.b_cols = p.H;
        j.N = p.H;
        j.k_blocks = j.wrap = 2 * p.I / 64;
        j.b_expert_rows = 2 * p.I;
        j.out = dx_sorted;
        j.out_f32 = problem->dx_dtype == MOE_DTYPE_FP32;
        jobs[n++] = j;
    }
    ProductJob w = {};
    w.a_rows = w.b_rows = cap;
    w.out_f32 = problem->dw_dtype == MOE_DTYPE_FP32;
    w.accumulate = problem->accumulate;
    if (dW13) {
        ProductJob j = w;
        j.a = dgu;
        j.a_rows = cap + 1LL;
        j.zero_in_a = 1;
        j.a_cols = 2LL * p.I;
        j.b = x_sorted;
        j.b_cols = p.H;
        j.M = 2 * p.I;
        j.N = p.H;
        j.out = dW13;
        jobs[n++] = j;
    }
    if (dW2) {
        ProductJob j = w;
        j.a = dy_sorted;
        j.a_cols = p.H;
        j.b = act;
        j.b_rows = cap + 1LL;
        j.b_cols = p.I;
        j.M = p.H;
        j.N = p.I;
        j.out = dW2;
        jobs[n++] = j;
    }
    return cuda_status(launch_products(jobs, n, {expert_offsets, nullptr, 0}, p.E, cap, err, sms, s));
}

moe_status_t moe_norm_backward_workspace_size(const moe_norm_problem_t *problem, size_t *bytes)
{
    if (!bytes)
        return MOE_ERR_NULL;
    const moe_status_t st = validate_norm(problem);
    if (st != MOE_OK)
        return st;
    *bytes = norm_layout(*problem).total;
    return MOE_OK;
}

moe_status_t moe_norm_backward(const moe_norm_problem_t *problem, const void *h, const void *w, const void *dx,
                               const void *dh_add, const int32_t *d_num_tokens, void *dh, void *dw, void *ws,
                               size_t ws_bytes, void *stream)
{
    moe_status_t st = validate_norm(problem);
    if (st != MOE_OK)
        return st;
    if (!h || !dx || !dh)
        return MOE_ERR_NULL;
    for (const void *q : {h, w, dx, dh_add, static_cast<const void *>(dh), static_cast<const void *>(dw)})
        if (!aligned(q, 16))
            return MOE_ERR_ALIGN;
    const moe_norm_problem_t &p = *problem;
    const NormGradLayout L = norm_layout(p);
    if ((st = check_ws(ws, ws_bytes, L.total)) != MOE_OK || (st = validate_device()) != MOE_OK)
        return st;
    NormGradArgs a = {};
    a.h = h;
    a.w = w;
    a.dx = dx;
    a.dh_add = dh_add;
    a.d_num_tokens = d_num_tokens;
    a.dh = dh;
    a.dw = dw;
    a.part = at<float>(ws, L.part);
    a.err = at<int32_t>(ws, 0);
    a.T_max = p.T_max;
    a.H = p.H;
    a.h_f32 = p.h_dtype == MOE_DTYPE_FP32;
    a.w_f32 = p.w_dtype == MOE_DTYPE_FP32;
    a.unit_offset = p.unit_offset;
    a.eps = p.eps;
    a.h_stride = p.h_stride ? p.h_stride : p.H;
    a.dx_stride = p.x_stride ? p.x_stride : p.H;
    a.add_stride = p.y_stride ? p.y_stride : p.H;
    a.out_stride = p.out_stride ? p.out_stride : p.H;
    return cuda_status(launch_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_route_backward_workspace_size(const moe_router_problem_t *problem, size_t *bytes)
{
    if (!bytes)
        return MOE_ERR_NULL;
    const moe_status_t st = check_route_grad(problem);
    if (st != MOE_OK)
        return st;
    *bytes = route_grad_layout(*problem).total;
    return MOE_OK;
}

moe_status_t moe_route_backward(const moe_router_problem_t *problem, int32_t dw_dtype, const void *x,
                                const void *w_router, const float *logits, const int32_t *topk_ids,
                                const float *d_weights, const float *d_logits_add, const int32_t *d_num_tokens,
                                void *dx, void *dw_router, float *d_logits, void *ws, size_t ws_bytes, void *stream)
{
    moe_status_t st = check_route_grad(problem);
    if (st != MOE_OK)
        return st;
    if (!is_dtype(dw_dtype))
        return MOE_ERR_SHAPE;
    if (!logits || !topk_ids || !d_weights || (dx && !w_router) || (dw_router && !x) || (!dx && !dw_router && !d_logits))
        return MOE_ERR_NULL;
    for (const void *q : {x, w_router, static_cast<const void *>(logits), static_cast<const void *>(topk_ids),
                          static_cast<const void *>(d_weights), static_cast<const void *>(d_logits_add),
                          static_cast<const void *>(dx), static_cast<const void *>(dw_router),
                          static_cast<const void *>(d_logits)})
        if (!aligned(q, 16))
            return MOE_ERR_ALIGN;
    const moe_router_problem_t &p = *problem;
    const RouteGradLayout L = route_grad_layout(p);
    if ((st = check_ws(ws, ws_bytes, L.total)) != MOE_OK || (st = validate_device()) != MOE_OK)
        return st;
    const RouteSplitK seg = route_segments(p);
    const int sms = device_sm_count(), Ep = (p.E + 63) / 64 * 64;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    RouteGradArgs a = {};
    a.logits = logits;
    a.ids = topk_ids;
    a.d_weights = d_weights;
    a.d_logits_add = d_logits_add;
    a.d_num_tokens = d_num_tokens;
    a.d_logits = d_logits;
    a.parts = at<void>(ws, L.parts);
    a.err = at<int32_t>(ws, 0);
    a.T_max = p.T_max;
    a.E = p.E;
    a.k = p.k;
    a.sigmoid = p.score == MOE_SCORE_SIGMOID;
    a.renormalize = p.renormalize;
    a.scale = p.scale;
    if (route_grad_few(a)) {
        RouteFewArgs f = {};
        f.x = static_cast<const __nv_bfloat16 *>(x);
        f.w = static_cast<const __nv_bfloat16 *>(w_router);
        f.dx = dx;
        f.dw = dw_router;
        f.dw_f32 = dw_dtype == MOE_DTYPE_FP32;
        f.H = p.H;
        return cuda_status(launch_route_grad_few(a, f, s));
    }
    if ((st = cuda_status(launch_route_grad(a, sms, s))) != MOE_OK)
        return st;
    ProductJob jobs[2];
    int n = 0;
    if (dw_router) {
        ProductJob j = {};
        j.rows_on_n = 1;
        j.a = x;
        j.a_rows = p.T_max;
        j.a_cols = p.H;
        j.b = a.parts;
        j.b_rows = p.T_max + 1LL;
        j.b_cols = 2LL * Ep;
        j.M = p.H;
        j.N = p.E;
        j.part_cols = Ep;
        j.out = seg.segments > 1 ? at<void>(ws, L.sums) : dw_router;
        j.out_f32 = seg.segments > 1 || dw_dtype == MOE_DTYPE_FP32;
        jobs[n++] = j;
    }
    if (dx) {
        ProductJob j = {};
        j.by_rows = 1;
        j.a = a.parts;
        j.a_rows = p.T_max;
        j.a_cols = 2LL * Ep;
        j.b = w_router;
        j.b_rows = p.E;
        j.b_cols = p.H;
        j.N = p.H;
        j.k_blocks = 2 * Ep / 64;
        j.wrap = Ep / 64;
        j.out = dx;
        jobs[n++] = j;
    }
    const ProductRows rows = {nullptr, d_num_tokens, seg.rows};
    if (n && (st = cuda_status(launch_products(jobs, n, rows, seg.segments, p.T_max, a.err, sms, s))) != MOE_OK)
        return st;
    if (dw_router && seg.segments > 1)
        return cuda_status(launch_sum_parts(at<float>(ws, L.sums), seg.segments, static_cast<size_t>(p.E) * p.H,
                                            dw_router, dw_dtype == MOE_DTYPE_FP32, sms, s));
    return MOE_OK;
}

}  // extern "C"
