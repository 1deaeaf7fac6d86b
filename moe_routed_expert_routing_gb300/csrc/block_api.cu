// block_api.cu -- C ABI of the block around the expert execution (declared
// and documented in include/moe.h): the norms, the router, and the whole
// layer for a few tokens. Host side only: validation (fails closed before any
// launch), workspace layout and launches.
#include <cmath>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr size_t kAlign = 256;
constexpr int kNormMaxHidden = 32768;
constexpr int kLayerMaxHidden = 16384;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool is_flag(int32_t v) { return v == 0 || v == 1; }

moe_status_t check_norm(const moe_norm_problem_t *p)
{
    if (!p)
        return MOE_ERR_NULL;
    if (p->T_max < 1 || p->T_max > (1 << 30) || p->H < 1 || p->H > kNormMaxHidden ||
        (p->h_dtype != MOE_DTYPE_BF16 && p->h_dtype != MOE_DTYPE_FP32) ||
        (p->w_dtype != MOE_DTYPE_BF16 && p->w_dtype != MOE_DTYPE_FP32) || !is_flag(p->unit_offset) ||
        !is_flag(p->norm_block) || p->gate < MOE_GATE_NONE || p->gate > MOE_GATE_ELEMENT)
        return MOE_ERR_SHAPE;
    if (!(p->eps > 0.f) || !std::isfinite(p->eps) || !std::isfinite(p->residual_scale))
        return MOE_ERR_SHAPE;
    if (p->H % 64 != 0)
        return MOE_ERR_ALIGN;
    for (const int64_t s : {p->h_stride, p->y_stride, p->x_stride, p->out_stride, p->gate_stride}) {
        if (s != 0 && (s < p->H || s > (int64_t(1) << 40)))
            return MOE_ERR_SHAPE;
        if (s % 8 != 0)
            return MOE_ERR_ALIGN;
    }
    return MOE_OK;
}

long long stride_of(int64_t s, int H) { return s ? s : H; }

NormArgs norm_args(const moe_norm_problem_t &p, const int32_t *d_num_tokens)
{
    NormArgs a = {};
    a.d_num_tokens = d_num_tokens;
    a.T_max = p.T_max;
    a.H = p.H;
    a.h_f32 = p.h_dtype == MOE_DTYPE_FP32;
    a.w_f32 = p.w_dtype == MOE_DTYPE_FP32;
    a.unit_offset = p.unit_offset;
    a.norm_block = p.norm_block;
    a.gate_kind = p.gate;
    a.eps = p.eps;
    a.scale = p.residual_scale;
    a.h_stride = stride_of(p.h_stride, p.H);
    a.y_stride = stride_of(p.y_stride, p.H);
    a.x_stride = stride_of(p.x_stride, p.H);
    a.out_stride = stride_of(p.out_stride, p.H);
    a.gate_stride = stride_of(p.gate_stride, p.H);
    return a;
}

moe_status_t check_router(const moe_router_problem_t *p)
{
    if (!p)
        return MOE_ERR_NULL;
    if (p->T_max < 1 || p->E < 1 || p->E > kMaxExperts || p->k < 1 || p->k > kMaxTopK || p->H < 1 ||
        (p->score != MOE_SCORE_SOFTMAX && p->score != MOE_SCORE_SIGMOID) || !is_flag(p->renormalize) ||
        !std::isfinite(p->scale))
        return MOE_ERR_SHAPE;
    if (p->n_group < 1 || p->n_group > 32 || p->E % p->n_group != 0 || p->topk_group < 1 ||
        p->topk_group > p->n_group || (p->group_top != 1 && p->group_top != 2) ||
        p->group_top > p->E / p->n_group || p->k > p->topk_group * (p->E / p->n_group))
        return MOE_ERR_SHAPE;
    if (p->n_group == 1 && p->group_top != 1)
        return MOE_ERR_SHAPE;
    if (static_cast<long long>(p->T_max) * p->k > (1LL << 28) || static_cast<long long>(p->T_max) * p->E > (1LL << 33) ||
        static_cast<long long>(p->E) * p->H > (1LL << 31))
        return MOE_ERR_SHAPE;
    if (p->H % 64 != 0)
        return MOE_ERR_ALIGN;
    return MOE_OK;
}

// Workspace of moe_route: the header (error word and counters), then the router's scratch.
struct RouteLayout {
    size_t part, total;
};

RouteLayout route_layout(const moe_router_problem_t &p)
{
    RouteLayout L;
    L.part = workspace_header_bytes();
    L.total = align_up(L.part + sizeof(float) * route_scratch_floats(p.T_max, p.E, p.H, false));
    return L;
}

RouteArgs route_args(const moe_router_problem_t &p)
{
    RouteArgs a = {};
    a.T_max = p.T_max;
    a.E = p.E;
    a.k = p.k;
    a.H = p.H;
    a.sigmoid = p.score == MOE_SCORE_SIGMOID;
    a.renormalize = p.renormalize;
    a.n_group = p.n_group;
    a.topk_group = p.topk_group;
    a.group_top = p.group_top;
    a.scale = p.scale;
    a.x_stride = p.H;
    return a;
}

moe_status_t check_layer(const moe_layer_problem_t *p)
{
    if (!p)
        return MOE_ERR_NULL;
    moe_status_t st = validate_problem(&p->experts);
    if (st != MOE_OK || (st = check_router(&p->router)) != MOE_OK || (st = check_norm(&p->norm)) != MOE_OK)
        return st;
    const moe_problem_t &e = p->experts;
    if (e.T_max > MOE_LAYER_MAX_TOKENS || e.T_max != p->router.T_max || e.T_max != p->norm.T_max ||
        e.E != p->router.E || e.k != p->router.k || e.H != p->router.H || e.H != p->norm.H || e.H > kLayerMaxHidden)
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

// Workspace of moe_layer: the one of moe_forward (header first), then the
// normalised rows (paired), the router's scratch and, for the one-kernel form of the
// experts, y and its row sums.
struct LayerLayout {
    size_t forward, x, part, y, sums, total;
};

LayerLayout layer_layout(const moe_layer_problem_t &p)
{
    LayerLayout L = {};
    L.forward = forward_workspace_bytes(paired_problem(p.experts));
    const size_t T = p.experts.T_max, H = p.experts.H;
    size_t o = align_up(L.forward);
    L.x = o;
    o = align_up(o + 2 * 2 * T * H);
    L.part = o;
    o = align_up(o + sizeof(float) * route_scratch_floats(p.experts.T_max, p.experts.E, p.experts.H, true));
    L.y = o;
    L.sums = align_up(o + sizeof(float) * T * H);
    if (p.experts.forward_form == MOE_FORWARD_ONE_KERNEL)
        o = align_up(L.sums + sizeof(float) * tail_sum_floats(p.experts.T_max, p.experts.H));
    L.total = o;
    return L;
}

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

// the way back into the residual stream: pointers as moe_norm_residual and moe_layer take them
moe_status_t check_residual(const moe_norm_problem_t &p, const void *h, const void *w_post, const void *gate,
                            const void *w_next, const void *h_out, const void *x_next)
{
    if (!h || !h_out || (p.gate != MOE_GATE_NONE && !gate))
        return MOE_ERR_NULL;
    for (const void *q : {h, w_post, gate, w_next, h_out, x_next})
        if (!aligned(q, 16))
            return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_norm(const moe_norm_problem_t *problem, const void *h, const void *w, const int32_t *d_num_tokens,
                      void *x, void *stream)
{
    moe_status_t st = check_norm(problem);
    if (st != MOE_OK)
        return st;
    if (!h || !x)
        return MOE_ERR_NULL;
    if (!aligned(h, 16) || !aligned(w, 16) || !aligned(x, 16))
        return MOE_ERR_ALIGN;
    if ((st = validate_device()) != MOE_OK)
        return st;
    NormArgs a = norm_args(*problem, d_num_tokens);
    a.h = h;
    a.w_next = w;
    a.x = x;
    return cuda_status(launch_norm(a, device_sm_count(), static_cast<cudaStream_t>(stream), true));
}

moe_status_t moe_norm_residual(const moe_norm_problem_t *problem, const void *h, const void *y, const void *w_post,
                               const void *gate, const void *w_next, const int32_t *d_num_tokens, void *h_out,
                               void *x_next, void *stream)
{
    moe_status_t st = check_norm(problem);
    if (st != MOE_OK)
        return st;
    if (!y)
        return MOE_ERR_NULL;
    if (!aligned(y, 16))
        return MOE_ERR_ALIGN;
    if ((st = check_residual(*problem, h, w_post, gate, w_next, h_out, x_next)) != MOE_OK)
        return st;
    if ((st = validate_device()) != MOE_OK)
        return st;
    NormArgs a = norm_args(*problem, d_num_tokens);
    a.h = h;
    a.y = y;
    a.w_post = w_post;
    a.gate = gate;
    a.w_next = w_next;
    a.h_out = h_out;
    a.x = x_next;
    return cuda_status(launch_norm(a, device_sm_count(), static_cast<cudaStream_t>(stream), true));
}

moe_status_t moe_route_workspace_size(const moe_router_problem_t *problem, size_t *bytes)
{
    if (!bytes)
        return MOE_ERR_NULL;
    const moe_status_t st = check_router(problem);
    if (st != MOE_OK)
        return st;
    *bytes = route_layout(*problem).total;
    return MOE_OK;
}

moe_status_t moe_route(const moe_router_problem_t *problem, const void *x, const void *w_router, const float *bias,
                       const int32_t *d_num_tokens, int32_t *topk_ids, float *topk_weights, float *logits, void *ws,
                       size_t ws_bytes, void *stream)
{
    moe_status_t st = check_router(problem);
    if (st != MOE_OK)
        return st;
    if (!x || !w_router || !topk_ids || !topk_weights)
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(bias, 16) || !aligned(topk_ids, 16) ||
        !aligned(topk_weights, 16) || !aligned(logits, 16))
        return MOE_ERR_ALIGN;
    const RouteLayout L = route_layout(*problem);
    if ((st = check_ws(ws, ws_bytes, L.total)) != MOE_OK || (st = validate_device()) != MOE_OK)
        return st;
    RouteArgs a = route_args(*problem);
    a.x = x;
    a.w = w_router;
    a.bias = bias;
    a.d_num_tokens = d_num_tokens;
    a.ids = topk_ids;
    a.weights = topk_weights;
    a.logits = logits;
    a.err = at<int32_t>(ws, 0);
    a.counters = at<int32_t>(ws, route_counters_offset());
    a.part = at<float>(ws, L.part);
    return cuda_status(launch_route(a, static_cast<cudaStream_t>(stream), true));
}

moe_status_t moe_layer_workspace_size(const moe_layer_problem_t *problem, size_t *bytes)
{
    if (!bytes)
        return MOE_ERR_NULL;
    const moe_status_t st = check_layer(problem);
    if (st != MOE_OK)
        return st;
    *bytes = layer_layout(*problem).total;
    return MOE_OK;
}

moe_status_t moe_layer(const moe_layer_problem_t *problem, const void *h, const void *w_pre, const void *w_router,
                       const float *bias, const void *W13, const void *W2, const void *w_post, const void *gate,
                       const void *w_next, const int32_t *d_num_tokens, int32_t *topk_ids, float *topk_weights,
                       int32_t *expert_offsets, int32_t *perm, void *h_out, void *x_next, void *ws, size_t ws_bytes,
                       void *stream)
{
    moe_status_t st = check_layer(problem);
    if (st != MOE_OK)
        return st;
    const moe_layer_problem_t &p = *problem;
    if (!w_router || !W13 || !W2 || !topk_ids || !topk_weights || !expert_offsets || !perm)
        return MOE_ERR_NULL;
    if ((st = check_residual(p.norm, h, w_post, gate, w_next, h_out, x_next)) != MOE_OK)
        return st;
    if (!aligned(w_pre, 16) || !aligned(w_router, 16) || !aligned(bias, 16) || !aligned(W13, 16) || !aligned(W2, 16) ||
        !aligned(topk_ids, 16) || !aligned(topk_weights, 16))
        return MOE_ERR_ALIGN;
    const LayerLayout L = layer_layout(p);
    if ((st = check_ws(ws, ws_bytes, L.total)) != MOE_OK || (st = validate_device()) != MOE_OK ||
        (st = check_forward(paired_problem(p.experts))) != MOE_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void *x = at<void>(ws, L.x);
    NormArgs n = norm_args(p.norm, d_num_tokens);
    n.h = h;
    n.w_post = w_post;
    n.gate = gate;
    n.w_next = w_next;
    n.h_out = h_out;
    n.x = x_next;
    // the norm, the router and the experts' rows: one kernel, or two
    RouteArgs r = route_args(p.router);
    r.x = h;
    r.x_stride = stride_of(p.norm.h_stride, p.norm.H);
    r.normed = 1;
    r.x_f32 = p.norm.h_dtype == MOE_DTYPE_FP32;
    r.w_f32 = p.norm.w_dtype == MOE_DTYPE_FP32;
    r.unit_offset = p.norm.unit_offset;
    r.w_pre = w_pre;
    r.eps = p.norm.eps;
    r.x_out = x;
    r.w = w_router;
    r.bias = bias;
    r.d_num_tokens = d_num_tokens;
    r.ids = topk_ids;
    r.weights = topk_weights;
    r.err = at<int32_t>(ws, 0);
    r.counters = at<int32_t>(ws, route_counters_offset());
    r.part = at<float>(ws, L.part);
    // a few routed slots: the router's last CTA dispatches them (the one-kernel
    // form of the experts dispatches by itself)
    r.one_kernel = p.experts.forward_form == MOE_FORWARD_ONE_KERNEL;
    const bool dispatched = p.experts.T_max <= kRouteJoinTokens &&
                            p.experts.T_max * p.experts.k <= kRouteDispatchSlots && !r.one_kernel;
    if (dispatched) {
        r.expert_offsets = expert_offsets;
        r.perm = perm;
        r.inv = forward_inv(paired_problem(p.experts), ws);
    }
    if ((st = cuda_status(launch_route(r, s, true))) != MOE_OK)
        return st;
    return enqueue_forward(p.experts, x, topk_ids, topk_weights, d_num_tokens, W13, W2, expert_offsets, perm,
                           at<void>(ws, L.y), ws, s, nullptr, &n, dispatched, at<float>(ws, L.sums));
}

}  // extern "C"
