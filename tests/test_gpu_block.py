"""The block around the experts on the GPU -- moe_norm, moe_norm_residual,
moe_route, moe_layer -- against plain 64-bit forms, at the sizes, types,
strides and masks where they can go wrong.

Tolerances, from the arithmetic:

* norms: fp32 with sums of at most a few hundred terms per thread and a tree
  over threads, so the mean of squares is within 8e-6 of its value and r
  within 4e-6; five more roundings of 6e-8. A bf16 output adds half a unit.
* logits: exact bf16 products, fp32 accumulation in steps of at least 16
  terms that may truncate: (H / 16 + 32) * 2^-23 of the sum of |products|.
* weights: the logits' error twice (numerator and sum), 1.2e-7 times the
  distance to the largest logit, and 2e-6 for the exponentials and sums.
* layer: x and h reach the MMAs with 16 bits, a relative 2^-17 each; their
  effect on a sum of thousands of terms stays below 2^-17 sqrt(terms) of its
  rms, so 1e-3 of y's rms bounds every element of y. It is carried through the
  gate, the scale and the norms.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_reference as ref
import oracle
import workloads as wlm
from parity import bf16_half_ulp

pytestmark = pytest.mark.gpu

NORM_REL = 5e-6
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def B():
    from moe_routed_expert_routing_gb300.build import build
    build()
    from moe_routed_expert_routing_gb300 import binding
    return binding


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, dtype, std=1.0, mean=0.0):
    return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(dtype)


def rows_apart(t, stride):
    """The same rows in a buffer whose rows lie `stride` apart, the rest filled with NaN."""
    if not stride or stride == t.shape[1]:
        return t.contiguous()
    buf = torch.full((t.shape[0], stride), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, : t.shape[1]] = t
    return buf[:, : t.shape[1]]


def check(got, want, tol, what):
    got = ref.f64(got)
    if not got.size:
        return
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{what}: error {err[worst]:.3e} at {worst}, allowed {np.broadcast_to(tol, err.shape)[worst]:.3e}"


def bf16_tol(want, rel=NORM_REL):
    return bf16_half_ulp(want) * (1 + 1e-3) + rel * np.abs(want) + 1e-30


# ------------------------------------------------------------------ norms

@pytest.mark.parametrize("T,H,h,w,stride,offset", [
    (1, 64, "bf16", "bf16", 0, False),
    (1, 7168, "bf16", "bf16", 0, False),
    (3, 2880, "fp32", "fp32", 2888, True),
    (17, 448, "bf16", "fp32", 512, False),
    (257, 4096, "fp32", "bf16", 0, False),
    (1031, 1536, "bf16", "bf16", 1544, True),
    (5, 8192, "bf16", None, 0, False),
    (2, 16384, "fp32", "bf16", 0, False),
    (2, 32768, "bf16", "fp32", 0, False),
    (3000, 128, "bf16", "bf16", 0, False),
])
def test_norm(B, T, H, h, w, stride, offset):
    g = gen(T + H)
    hh = rows_apart((randn(g, (T, H), torch.float32) * torch.exp(randn(g, (T, 1), torch.float32, 2.0))).to(DT[h]), stride)
    ww = None if w is None else randn(g, (H,), DT[w], 0.2, 0.0 if offset else 1.0)
    x = torch.full((T, stride or H), 7.0, dtype=torch.bfloat16, device="cuda")
    p = B.NormProblem.make(T, H, h_dtype=DT[h], w_dtype=DT[w or "bf16"], eps=1e-5, unit_offset=offset,
                           h_stride=stride, x_stride=stride)
    B.moe_norm(p, hh, ww, x[:, :H])
    want = ref.norm(ref.f64(hh), ref.f64(ww), 1e-5, offset)
    check(x[:, :H], want, bf16_tol(want), "x")
    if stride:
        assert (x[:, H:] == 7.0).all()          # the gap between rows is not written


def test_norm_zero_row_and_device_token_count(B):
    T, H = 9, 512
    h = randn(gen(1), (T, H), torch.bfloat16)
    h[2] = 0
    h[3] = 1e-30
    p = B.NormProblem.make(T, H, eps=1e-6)
    for n, rows in [(None, T), (5, 5), (0, 0), (-3, 0), (100, T)]:
        x = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
        d = None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda")
        B.moe_norm(p, h, None, x, d_num_tokens=d)
        want = ref.norm(ref.f64(h))
        check(x[:rows], want[:rows], bf16_tol(want[:rows]), "x")
        assert (x[rows:] == 7.0).all()


def residual_tol(h_new, step, dtype):
    tol = 2.0 ** -22 * np.abs(h_new) + (NORM_REL + 5e-7) * np.abs(step) + 2.0 ** -23 * (np.abs(h_new) + np.abs(step))
    return tol + (bf16_half_ulp(h_new) * (1 + 1e-3) if dtype == "bf16" else 0.0) + 1e-30


@pytest.mark.parametrize("T,H,h,w,post,gate,nxt,stride,in_place", [
    (1, 64, "bf16", "bf16", True, 0, True, 0, False),
    (1, 7168, "bf16", "bf16", True, 0, True, 0, True),
    (7, 7168, "fp32", "bf16", True, 1, False, 0, False),
    (13, 2880, "bf16", "fp32", False, 2, True, 2944, False),
    (33, 448, "fp32", "fp32", True, 3, True, 456, True),
    (100, 4096, "bf16", "bf16", False, 0, False, 0, False),
    (1029, 1024, "fp32", "bf16", True, 2, True, 0, False),
    (3, 16384, "bf16", "bf16", True, 1, True, 0, True),
    (2, 32768, "fp32", "fp32", True, 3, True, 0, False),
    (640, 192, "bf16", "fp32", True, 3, False, 0, True),
])
def test_norm_residual(B, T, H, h, w, post, gate, nxt, stride, in_place):
    g = gen(T * 3 + H)
    hh = rows_apart(randn(g, (T, H), DT[h], 2.0), stride)
    y = rows_apart((randn(g, (T, H), torch.float32) * torch.exp(randn(g, (T, 1), torch.float32, 2.0))).bfloat16(), stride)
    w_post = randn(g, (H,), DT[w], 0.2, 1.0) if post else None
    w_next = randn(g, (H,), DT[w], 0.2, 1.0) if nxt else None
    gt = {0: None, 1: randn(g, (H,), DT[w], 0.5), 2: randn(g, (T,), torch.float32),
          3: rows_apart(randn(g, (T, H), torch.bfloat16), stride)}[gate]
    p = B.NormProblem.make(T, H, h_dtype=DT[h], w_dtype=DT[w], eps=1e-6, norm_block=post, gate=gate, residual_scale=0.3,
                           h_stride=stride, y_stride=stride, x_stride=stride, out_stride=stride, gate_stride=stride)
    want, step = ref.residual(ref.f64(hh), ref.f64(y), ref.f64(w_post), post, ref.f64(gt), gate, 0.3)
    out = hh if in_place else rows_apart(torch.zeros((T, H), dtype=DT[h], device="cuda"), stride)
    x_next = rows_apart(torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), stride) if nxt else None
    B.moe_norm_residual(p, hh, y, out, w_post=w_post, gate=gt, w_next=w_next, x_next=x_next)
    tol = residual_tol(want, step, h)
    check(out, want, tol, "h_out")
    if nxt:
        nx = ref.norm(want, ref.f64(w_next))
        moved = residual_tol(want, step, "fp32") * ref.rms_scale(want, 1e-6) * np.abs(ref.f64(w_next))
        check(x_next, nx, bf16_tol(nx) + moved, "x_next")


def test_norm_residual_token_count_and_unweighted(B):
    T, H = 11, 256
    g = gen(3)
    h, y = randn(g, (T, H), torch.bfloat16), randn(g, (T, H), torch.bfloat16)
    y[4] = 0                                   # a row whose experts were all dropped
    p = B.NormProblem.make(T, H, norm_block=True)
    out = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    nxt = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_norm_residual(p, h, y, out, x_next=nxt, d_num_tokens=torch.tensor([6], dtype=torch.int32, device="cuda"))
    want, step = ref.residual(ref.f64(h), ref.f64(y), None, True)
    check(out[:6], want[:6], residual_tol(want, step, "bf16")[:6], "h_out")
    assert torch.equal(out[4], h[4])
    n = ref.norm(want)
    check(nxt[:6], n[:6], (bf16_tol(n) + residual_tol(want, step, "fp32") * ref.rms_scale(want, 1e-6))[:6], "x_next")
    assert (out[6:] == 7.0).all() and (nxt[6:] == 7.0).all()


# ------------------------------------------------------------------ router

def grid_inputs(g, T, E, H):
    """Inputs whose logits are exact in fp32 in any order of summation: multiples of 2^-3 with small sums."""
    x = torch.randint(-2, 3, (T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randint(-1, 2, (E, H), generator=g, device="cuda") * (torch.rand((E, H), generator=g, device="cuda") < 64.0 / H) / 8).to(torch.bfloat16)
    return x, w


def run_route(B, p, x, w, bias=None, logits=None, T_dev=None, ws=None):
    ids = torch.full((p.T_max, p.k), -9, dtype=torch.int32, device="cuda")
    wt = torch.full((p.T_max, p.k), -9.0, dtype=torch.float32, device="cuda")
    ws = torch.zeros(B.moe_route_workspace_size(p), dtype=torch.uint8, device="cuda") if ws is None else ws
    d = None if T_dev is None else torch.tensor([T_dev], dtype=torch.int32, device="cuda")
    B.moe_route(p, x, w, ids, wt, ws, bias=bias, logits=logits, d_num_tokens=d)
    return ids, wt, ws


ROUTE_SHAPES = [(1, 1, 1, 64), (1, 384, 6, 7168), (2, 7, 7, 128), (9, 33, 4, 192), (31, 130, 8, 2880), (64, 256, 8, 1024),
                (65, 128, 64, 512), (100, 1000, 10, 448), (129, 384, 6, 1536), (300, 512, 8, 512), (513, 96, 2, 4096),
                (300, 128, 64, 128), (200, 200, 33, 64), (192, 48, 3, 128), (193, 48, 3, 128), (150, 1024, 4, 64),
                                (1025, 1024, 16, 256), (2500, 64, 8, 320)]


@pytest.mark.parametrize("T,E,k,H", ROUTE_SHAPES)
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", False)])
def test_route_exact_logits_and_ties(B, T, E, k, H, score, renorm):
    x, w = grid_inputs(gen(T + E), T, E, H)
    logits = torch.empty((T, E), device="cuda")
    p = B.RouterProblem.make(T, E, k, H, score=int(score == "sigmoid"), renormalize=renorm, scale=1.5)
    ids, wt, ws = run_route(B, p, x, w, logits=logits)
    want_l = ref.f64(x) @ ref.f64(w).T
    assert np.array_equal(ref.f64(logits), want_l)
    want_ids, want_w, _ = ref.route(want_l, k, score, renorm, scale=1.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    spread = want_l.max(axis=1, keepdims=True) - want_l.min(axis=1, keepdims=True)
    check(wt, want_w, np.abs(want_w) * (4e-6 + 2.4e-7 * spread) + 1e-37, "weights")
    assert B.moe_last_device_error(ws) == 0
    again, wt2, _ = run_route(B, p, x, w, ws=ws)      # no logits asked for, the same workspace again
    assert torch.equal(again, ids) and torch.equal(wt2, wt)


@pytest.mark.parametrize("T", [2, 200])
@pytest.mark.parametrize("E,k", [(100, 8), (70, 40)])
def test_route_equal_logits(B, T, E, k):
    """All experts equal: the lowest k, in order; and rows where only a few differ."""
    H = 64
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((E, H), dtype=torch.bfloat16, device="cuda")
    w[50:53, 0] = 1.0
    x[0] = 0
    x[-1] = -1
    for score in (0, 1):
        p = B.RouterProblem.make(T, E, k, H, score=score)
        ids, wt, _ = run_route(B, p, x, w)
        want_ids, want_w, _ = ref.route(ref.f64(x) @ ref.f64(w).T, k, ("softmax", "sigmoid")[score])
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        check(wt, want_w, np.abs(want_w) * 4e-6, "weights")


@pytest.mark.parametrize("T,E,k,H", [(1, 384, 6, 7168), (40, 256, 8, 2880), (515, 384, 6, 7168), (2048, 128, 8, 4096),
                                     (77, 1024, 8, 448)])
def test_route_real_logits(B, T, E, k, H):
    g = gen(E + T)
    x = randn(g, (T, H), torch.bfloat16)
    w = randn(g, (E, H), torch.bfloat16, H ** -0.5)
    logits = torch.empty((T, E), device="cuda")
    p = B.RouterProblem.make(T, E, k, H)
    ids, wt, _ = run_route(B, p, x, w, logits=logits)
    want = ref.f64(x) @ ref.f64(w).T
    tol = (H / 16 + 32) * 2.0 ** -23 * (np.abs(ref.f64(x)) @ np.abs(ref.f64(w)).T)
    check(logits, want, tol, "logits")
    # the selection on the kernel's own logits is exact
    got_l = ref.f64(logits)
    want_ids, want_w, _ = ref.route(got_l, k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    spread = got_l.max(axis=1, keepdims=True) - got_l.min(axis=1, keepdims=True)
    check(wt, want_w, np.abs(want_w) * (4e-6 + 2.4e-7 * spread), "weights")


@pytest.mark.parametrize("T,E,k,H,score,groups,keep,top,bias", [
    (1, 256, 8, 7168, "sigmoid", 8, 4, 2, True),
    (61, 256, 8, 512, "sigmoid", 8, 4, 2, True),
    (200, 160, 6, 256, "softmax", 8, 3, 1, False),
    (33, 1024, 16, 128, "sigmoid", 32, 5, 2, True),
    (150, 64, 4, 192, "softmax", 1, 1, 1, True),
    (19, 36, 3, 64, "sigmoid", 4, 1, 2, False),
    (700, 384, 8, 256, "sigmoid", 2, 1, 1, True),
    (160, 32, 5, 64, "softmax", 32, 7, 1, False),
    (12, 30, 2, 64, "softmax", 10, 3, 2, True),
    (260, 512, 12, 128, "sigmoid", 16, 6, 1, True),
])
def test_route_groups_and_bias(B, T, E, k, H, score, groups, keep, top, bias):
    g = gen(E * 7 + T)
    x, w = grid_inputs(g, T, E, H)
    b = randn(g, (E,), torch.float32, 0.1) if bias else None
    p = B.RouterProblem.make(T, E, k, H, score=int(score == "sigmoid"), n_group=groups, topk_group=keep,
                             group_top=top, scale=2.5)
    ids, wt, _ = run_route(B, p, x, w, bias=b)
    want_l = ref.f64(x) @ ref.f64(w).T
    want_ids, want_w, margin = ref.route(want_l, k, score, True, ref.f64(b), groups, keep, top, 2.5)
    sure = margin > 2e-6              # keys are fp32 sums of a score and a bias
    assert sure.mean() > 0.8
    assert np.array_equal(ids.cpu().numpy()[sure], want_ids[sure])
    check(wt[torch.from_numpy(sure).cuda()], want_w[sure], np.abs(want_w[sure]) * 1e-5 + 1e-37, "weights")


@pytest.mark.parametrize("T", [1, 5, 120, 200])
def test_route_masked_experts(B, T):
    """Experts switched off by a bias of -inf, down to fewer than k, then none."""
    E, k, H = 40, 6, 128
    x, w = grid_inputs(gen(9), T, E, H)
    for on in (E, 7, 6, 3, 1, 0):
        bias = torch.full((E,), float("-inf"), device="cuda")
        bias[torch.randperm(E, generator=torch.Generator().manual_seed(on))[:on].cuda()] = 0.0
        for score in (0, 1):
            for renorm in (True, False):
                p = B.RouterProblem.make(T, E, k, H, score=score, renormalize=renorm)
                ids, wt, ws = run_route(B, p, x, w, bias=bias)
                want_ids, want_w, margin = ref.route(ref.f64(x) @ ref.f64(w).T, k, ("softmax", "sigmoid")[score], renorm,
                                                     ref.f64(bias))
                sure = margin > 2e-7
                assert np.array_equal(ids.cpu().numpy()[sure], want_ids[sure])
                check(wt[torch.from_numpy(sure).cuda()], want_w[sure], np.abs(want_w[sure]) * 1e-5 + 1e-37, "weights")
                assert (ids.cpu().numpy()[:, min(on, k):] == -1).all() and (wt[:, min(on, k):] == 0).all()
                assert B.moe_last_device_error(ws) == 0


def test_route_bias_that_makes_all_keys_equal_leaves_nothing_behind(B):
    """Many tokens, keys equal by the bias: the lowest experts, for every token and in every repeat."""
    T, E, k, H = 300, 200, 8, 64
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((E, H), dtype=torch.bfloat16, device="cuda")
    bias = torch.full((E,), 3.0, device="cuda")
    p = B.RouterProblem.make(T, E, k, H, score=1)
    ws = None
    for _ in range(3):
        ids, wt, ws = run_route(B, p, x, w, bias=bias, ws=ws)
        assert (ids == torch.arange(k, dtype=torch.int32, device="cuda")).all()
        assert (wt - 1.0 / k).abs().max() < 1e-6


@pytest.mark.parametrize("T", [3, 300])
def test_route_logits_that_are_not_numbers(B, T):
    """NaN and +inf logits are never chosen and set the error bit; -inf logits are just never chosen."""
    E, k, H = 70, 4, 128
    x, w = grid_inputs(gen(5), T, E, H)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    w[10, 0] = float("-inf")
    p = B.RouterProblem.make(T, E, k, H)
    ids, wt, ws = run_route(B, p, x, w)
    l = ref.f64(x) @ np.nan_to_num(ref.f64(w), neginf=0.0).T
    l[:, 10] = -np.inf
    want_ids, want_w, _ = ref.route(l, k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert B.moe_last_device_error(ws) == 0
    w[3, 0] = float("nan")
    w[60, 0] = float("inf")
    ids, wt, ws = run_route(B, p, x, w)
    l[:, [3, 60]] = -np.inf
    want_ids, want_w, _ = ref.route(l, k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    check(wt, want_w, np.abs(want_w) * 1e-5 + 1e-37, "weights")
    assert B.moe_last_device_error(ws) == B.MOE_DEVERR_BAD_LOGIT
    # a token of NaN: every slot dropped
    x[1] = float("nan")
    ids, wt, ws = run_route(B, p, x, w)
    assert (ids[1] == -1).all() and (wt[1] == 0).all()
    assert np.array_equal(np.delete(ids.cpu().numpy(), 1, 0), np.delete(want_ids, 1, 0))


@pytest.mark.parametrize("scale_up", [40.0, 400.0])
def test_route_far_apart_logits(B, scale_up):
    """Scores that underflow or saturate keep the logits' order and their ratios."""
    T, E, k, H = 6, 48, 8, 256
    x, w = grid_inputs(gen(2), T, E, H)
    w = (w.float() * scale_up).bfloat16()
    l = ref.f64(x) @ ref.f64(w).T
    for score in (0, 1):
        for shift in (0.0, -200.0):
            ww, xx = w.clone(), x.clone()
            xx[:, 0], ww[:, 0] = 1.0, shift
            ll = ref.f64(xx) @ ref.f64(ww).T
            p = B.RouterProblem.make(T, E, k, H, score=score)
            ids, wt, ws = run_route(B, p, xx, ww)
            want_ids, want_w, _ = ref.route(ll, k, ("softmax", "sigmoid")[score])
            assert np.array_equal(ids.cpu().numpy(), want_ids)
            check(wt, want_w, np.abs(want_w) * (4e-6 + 2.4e-7 * np.abs(ll).max()) + 1e-37, "weights")


@pytest.mark.parametrize("T", [6, 400])
def test_route_device_token_count_in_a_graph(B, T):
    E, k, H = 72, 5, 192
    x, w = grid_inputs(gen(11), T, E, H)
    p = B.RouterProblem.make(T, E, k, H)
    full, wfull, ws = run_route(B, p, x, w)
    ids = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    wt = torch.full((T, k), -9.0, device="cuda")
    logits = torch.full((T, E), -9.0, device="cuda")
    d = torch.tensor([0], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_route(p, x, w, ids, wt, ws, logits=logits, d_num_tokens=d)
    for n in (T - 2, 1, 0, T):
        ids.fill_(-9)
        wt.fill_(-9.0)
        logits.fill_(-9.0)
        d.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids[:n], full[:n]) and torch.equal(wt[:n], wfull[:n])
        assert (ids[n:] == -9).all() and (wt[n:] == -9.0).all() and (logits[n:] == -9.0).all()


# ------------------------------------------------------------------- layer

class LayerCase:
    """Inputs of one layer, in bf16, and the 64-bit form of its pieces."""

    def __init__(self, B, T, E, k, H, I, seed=0, h="bf16", w="bf16", score=0, bias=False, groups=(1, 1, 1), post=True,
                 gate=0, nxt=True, scale=0.7, layout=0, form=0, path=0, offset=False, stride=0):
        g = gen(seed + T + E)
        self.B, self.T, self.k, self.post, self.gate_kind, self.scale, self.offset = B, T, k, post, gate, scale, offset
        self.h = rows_apart(randn(g, (T, H), DT[h], 2.0), stride)
        self.w_pre = randn(g, (H,), DT[w], 0.2, 0.0 if offset else 1.0)
        self.w_router = randn(g, (E, H), torch.bfloat16, H ** -0.5)
        self.bias = randn(g, (E,), torch.float32, 0.05) if bias else None
        self.W13 = randn(g, (E, 2 * I, H), torch.bfloat16, H ** -0.5)
        self.W2 = randn(g, (E, H, I), torch.bfloat16, I ** -0.5)
        self.w_post = randn(g, (H,), DT[w], 0.2, 1.0) if post else None
        self.w_next = randn(g, (H,), DT[w], 0.2, 1.0) if nxt else None
        self.gate = {0: None, 1: randn(g, (H,), DT[w], 0.5), 2: randn(g, (T,), torch.float32),
                     3: randn(g, (T, H), torch.bfloat16)}[gate]
        self.norm = B.NormProblem.make(T, H, h_dtype=DT[h], w_dtype=DT[w], norm_block=post, gate=gate,
                                       residual_scale=scale, unit_offset=offset, h_stride=stride)
        self.router = B.RouterProblem.make(T, E, k, H, score=score, n_group=groups[0], topk_group=groups[1],
                                           group_top=groups[2])
        self.experts = B.Problem.make(T, E, k, H, I, weight_layout=layout, forward_form=form, path=path)
        self.p = B.LayerProblem.make(self.experts, self.router, self.norm)
        self.args13, self.args2 = self.W13, self.W2
        self.ref13, self.ref2 = ref.f64(self.W13), ref.f64(self.W2)
        if layout == B.MOE_WEIGHTS_PACKED:
            self.args13, self.args2 = B.moe_pack_weights(self.experts, self.W13, self.W2)
        if layout == B.MOE_WEIGHTS_MXFP8:
            self.args13, self.args2 = B.moe_quantize_weights(self.experts, self.W13, self.W2)
            self.ref13, self.ref2 = (oracle.bf16_bits_to_f32(oracle.mx_dequantize(*oracle.mx_quantize(wlm.bf16_bits(w)))).astype(np.float64)
                                     for w in (self.W13, self.W2))
        self.ws = torch.zeros(B.moe_layer_workspace_size(self.p), dtype=torch.uint8, device="cuda")
        self.h_type = h

    def run(self, T_dev=None, h_out=None, d=None):
        B, p = self.B, self.experts
        o = {"ids": torch.full((p.T_max, p.k), -9, dtype=torch.int32, device="cuda"),
             "weights": torch.full((p.T_max, p.k), -9.0, device="cuda"),
             "offsets": torch.full((p.E + 1,), -9, dtype=torch.int32, device="cuda"),
             "perm": torch.full((p.T_max * p.k,), -9, dtype=torch.int32, device="cuda"),
             "h": torch.full((p.T_max, p.H), 7.0, dtype=self.h.dtype, device="cuda") if h_out is None else h_out,
             "x_next": None if self.w_next is None else torch.full((p.T_max, p.H), 7.0, dtype=torch.bfloat16, device="cuda")}
        if T_dev is not None:
            d = torch.tensor([T_dev], dtype=torch.int32, device="cuda")
        self.call(o, d)
        return o

    def call(self, o, d=None):
        self.B.moe_layer(self.p, self.h, self.w_pre, self.w_router, self.args13, self.args2, o["ids"], o["weights"],
                         o["offsets"], o["perm"], o["h"], self.ws, bias=self.bias, w_post=self.w_post, gate=self.gate,
                         w_next=self.w_next, x_next=o["x_next"], d_num_tokens=d)

    def verify(self, o, T=None, h_in=None):
        T = self.T if T is None else T
        r = self.router
        h = ref.f64(self.h if h_in is None else h_in)
        v = ref.norm(h, ref.f64(self.w_pre), 1e-6, self.offset)
        logits = v @ ref.f64(self.w_router).T
        ids, w, margin = ref.route(logits, self.k, ("softmax", "sigmoid")[r.score], True, ref.f64(self.bias), r.n_group,
                                   r.topk_group, r.group_top)
        # logits of the unrounded rows: 3e-6 of r and of the products' split, 2^-21 accumulation of |v||w| sums
        lt = float((1e-5 * (np.abs(v) @ np.abs(ref.f64(self.w_router)).T)).max())
        sure = np.flatnonzero((margin > 2 * lt) & (np.arange(len(margin)) < T))
        assert len(sure) >= 0.5 * T
        got = o["ids"].cpu().numpy()
        assert np.array_equal(got[sure], ids[sure])
        check(o["weights"][torch.from_numpy(sure).cuda()], w[sure], np.abs(w[sure]) * (2 * lt + 1e-5), "weights")
        # the dispatch tables follow the ids the call returns
        _, off, perm, _, _ = oracle.dispatch(got[:T], self.experts.E)
        assert np.array_equal(o["offsets"].cpu().numpy(), off)
        assert np.array_equal(o["perm"].cpu().numpy()[: off[-1]], perm[: off[-1]])
        y = ref.experts(v[:T], got[:T], ref.f64(o["weights"])[:T], self.ref13, self.ref2)
        gt = ref.gate_rows(ref.f64(self.gate), self.gate_kind)
        gt = gt[:T] if self.gate_kind >= 2 else gt
        y_tol = 1e-3 * np.sqrt((y ** 2).mean()) if T else 0.0
        h_new, step = ref.residual(h[:T], y, ref.f64(self.w_post), self.post,
                                   None if self.gate is None else (ref.f64(self.gate)[:T] if self.gate_kind >= 2 else ref.f64(self.gate)),
                                   self.gate_kind, self.scale, 1e-6, self.offset)
        moved = y_tol * np.abs(gt) * self.scale
        if self.post:
            wp = np.abs(ref.f64(self.w_post) + (1.0 if self.offset else 0.0))
            # the norm's own scale moves by the rows' mean error, far below the largest
            moved = 1.2 * moved * ref.rms_scale(y, 1e-6) * wp + 1e-4 * np.abs(step)
        tol = moved + residual_tol(h_new, step, self.h_type)
        check(o["h"][:T], h_new, tol, "h_out")
        if self.w_next is not None:
            wn = ref.f64(self.w_next) + (1.0 if self.offset else 0.0)
            n = ref.norm(h_new, ref.f64(self.w_next), 1e-6, self.offset)
            t2 = (moved + residual_tol(h_new, step, "fp32")) * ref.rms_scale(h_new, 1e-6) * np.abs(wn) + 1e-4 * np.abs(n)
            check(o["x_next"][:T], n, bf16_tol(n) + t2, "x_next")
        assert (o["h"][T:] == 7.0).all() and (o["ids"][T:] == -9).all() and (o["weights"][T:] == -9.0).all()
        assert self.B.moe_last_device_error(self.ws) == 0


LAYERS = [
    dict(T=1, E=64, k=6, H=1024, I=512),
    dict(T=1, E=1, k=1, H=64, I=64, post=False, nxt=False),
    dict(T=2, E=384, k=6, H=448, I=192, h="fp32", gate=1),
    dict(T=5, E=40, k=3, H=2880, I=320, score=1, bias=True, gate=2),
    dict(T=8, E=64, k=4, H=512, I=256, post=False, gate=3, w="fp32"),
    dict(T=16, E=16, k=8, H=768, I=128, offset=True),
    dict(T=33, E=128, k=8, H=1024, I=192, score=1, bias=True, groups=(8, 4, 2), gate=1),
    dict(T=64, E=32, k=4, H=512, I=128, h="fp32", w="fp32", stride=520),
    dict(T=100, E=24, k=2, H=320, I=256, gate=2),
    dict(T=128, E=8, k=2, H=256, I=512, post=False),
    dict(T=128, E=1024, k=2, H=128, I=64),
    dict(T=3, E=4, k=2, H=16384, I=64, gate=1),
    dict(T=9, E=32, k=3, H=8256, I=128, h="fp32", score=1),
    dict(T=40, E=300, k=64, H=64, I=64),
    dict(T=2, E=100, k=64, H=64, I=64, nxt=False),
]


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "T{T}E{E}k{k}H{H}I{I}".format(**c))
def test_layer(B, case):
    c = LayerCase(B, **case)
    o = c.run()
    c.verify(o)
    o2 = c.run()                       # counters are back at zero, results repeat bit for bit
    for key in ("ids", "weights", "h", "x_next"):
        if o[key] is not None:
            assert torch.equal(o[key], o2[key]), key


@pytest.mark.parametrize("layout", [1, 2])
@pytest.mark.parametrize("T", [1, 13, 100])
def test_layer_packed_and_mxfp8_weights(B, layout, T):
    c = LayerCase(B, T=T, E=32, k=4, H=512, I=256, layout=layout, gate=1)
    c.verify(c.run())


@pytest.mark.parametrize("T,layout", [(1, 0), (4, 1), (8, 2), (16, 0)])
def test_layer_two_kernel_form(B, T, layout):
    one = LayerCase(B, T=T, E=64, k=4, H=512, I=256, layout=layout, form=2, gate=1)
    o = one.run()
    one.verify(o)
    o2 = one.run()
    assert torch.equal(o["h"], o2["h"])


@pytest.mark.parametrize("path", [1, 2, 3])
def test_layer_every_expert_path(B, path):
    c = LayerCase(B, T=48, E=8, k=2, H=512, I=256, path=path)
    c.verify(c.run())


def test_layer_in_place_and_device_token_count_in_a_graph(B):
    c = LayerCase(B, T=24, E=32, k=4, H=512, I=128, gate=2)
    h0 = c.h.clone()
    full = c.run()
    d = torch.tensor([24], dtype=torch.int32, device="cuda")
    o = c.run(d=d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(o, d)
    for n in (24, 1, 17, 0):
        for key, fill in (("h", 7.0), ("x_next", 7.0), ("ids", -9), ("weights", -9.0)):
            o[key].fill_(fill)
        d.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        for key, fill in (("h", 7.0), ("x_next", 7.0), ("ids", -9), ("weights", -9.0)):
            assert torch.equal(o[key][:n], full[key][:n]) and (o[key][n:] == fill).all(), (key, n)
    o = c.run(h_out=c.h)               # in place
    assert torch.equal(o["h"], full["h"]) and torch.equal(o["x_next"], full["x_next"])
    assert not torch.equal(h0, c.h)


@pytest.mark.parametrize("T,form", [(1, 0), (2, 0), (3, 0), (2, 2)])
def test_layer_device_token_count_of_the_smallest(B, T, form):
    c = LayerCase(B, T=T, E=32, k=4, H=256, I=128, form=form)
    full = c.run()
    c.verify(full)
    for n in range(T + 1):
        o = c.run(T_dev=n)
        for key, fill in (("h", 7.0), ("x_next", 7.0), ("ids", -9), ("weights", -9.0)):
            assert torch.equal(o[key][:n], full[key][:n]) and (o[key][n:] == fill).all(), (key, n)
        off = o["offsets"].cpu().numpy()
        assert off[0] == 0 and off[-1] == n * 4 and (np.diff(off) >= 0).all()
    assert B.moe_last_device_error(c.ws) == 0


@pytest.mark.parametrize("T,form", [(2, 0), (6, 0), (6, 2), (40, 0)])
def test_layer_with_a_row_of_nan(B, T, form):
    """A NaN row is routed nowhere, sets the error bit and leaves the other rows as they are."""
    c = LayerCase(B, T=T, E=64, k=4, H=256, I=128, form=form)
    good = c.run()
    assert B.moe_last_device_error(c.ws) == 0
    c.h[1] = float("nan")
    o = c.run()
    assert B.moe_last_device_error(c.ws) == B.MOE_DEVERR_BAD_LOGIT
    rest = [t for t in range(T) if t != 1]
    assert (o["ids"][1] == -1).all() and (o["weights"][1] == 0).all() and torch.isnan(o["h"][1].float()).all()
    for key in ("ids", "weights", "h", "x_next"):
        assert torch.equal(o[key][rest], good[key][rest]), key
    assert int(o["offsets"][-1]) == (T - 1) * 4


def test_layer_matches_its_pieces(B):
    """The layer and moe_norm, moe_route, moe_forward, moe_norm_residual in turn: the same experts
    (away from near ties), outputs within bf16 roundings of x and y."""
    c = LayerCase(B, T=20, E=32, k=4, H=1024, I=256)
    o = c.run()
    T, H, k, E = 20, 1024, 4, 32
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    B.moe_norm(c.norm, c.h, c.w_pre, x)
    ids, wt, _ = run_route(B, c.router, x, c.w_router)
    same = (ids == o["ids"]).all(1)
    assert same.float().mean() > 0.8
    bufs = B.Buffers(c.experts)
    B.moe_forward(c.experts, x, ids, wt, c.W13, c.W2, bufs.expert_offsets, bufs.perm, bufs.out, bufs.ws)
    h_out, x_next = torch.empty_like(c.h), torch.empty_like(x)
    B.moe_norm_residual(c.norm, c.h, bufs.out, h_out, w_post=c.w_post, w_next=c.w_next, x_next=x_next)
    a, b = ref.f64(h_out[same]), ref.f64(o["h"][same])
    # the pieces round x, h (of gate times up, each moved by x) and y to bf16, 1.7e-3 of rms each: with the gate and
    # up counted apart, five deviations of four such roundings; and each side rounds its output, half a unit
    step = b - ref.f64(c.h[same])
    bound = 5 * 2 * 1.7e-3 * np.sqrt((step ** 2).mean()) * np.abs(ref.f64(c.w_post)).max()
    assert (np.abs(a - b) <= bound + 2 * bf16_half_ulp(np.maximum(np.abs(a), np.abs(b)))).all()


def test_layer_on_a_side_stream(B):
    c = LayerCase(B, T=6, E=32, k=4, H=512, I=128)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run()
    s.synchronize()
    assert torch.equal(want["h"], got["h"]) and torch.equal(want["ids"], got["ids"])
