"""The gradients' kernels where a block does several units of work in a row, an
expert holds several slots of the router's one-kernel form, and what they report.
Tolerances as in test_gpu_backward.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import backward_reference as back
import block_reference as ref
from test_gpu_backward import (B, BF, F32, U, Step, block_case, check, count, empty, expert_inputs, expert_problem,  # noqa: F401
                               gen, randn, route_inputs, run_experts, run_route)

pytestmark = pytest.mark.gpu

PAIRS = 76          # CTA pairs of a GB300 at most


def act_units(counts, I, tile_rows):
    return sum((n + tile_rows - 1) // tile_rows for n in counts) * ((I + 127) // 128)


def check_experts(out, x, dy, W13, W2, bounds):
    n = int(bounds[-1])
    want, tol = back.experts(ref.f64(x[:n]), ref.f64(dy[:n]), ref.f64(W13), ref.f64(W2), bounds)
    check(out["dx_sorted"][:n], want["dx"], tol["dx"], "dx")
    check(out["dW13"], want["dW13"], tol["dW13"], "dW13")
    check(out["dW2"], want["dW2"], tol["dW2"], "dW2")
    assert (out["dx_sorted"][n:] == 7.0).all()


MIXED = [1, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 255, 256, 257, 0, 320]


@pytest.mark.parametrize("counts,H,I", [
    # over 128 rows an expert on average: whole tiles
    ([300, 129, 700, 40], 192, 2944),
    ([300, 0, 513, 64, 257], 256, 2560),
    # 25 to 128: tiles in halves of 32 and 64 rows beside whole ones, an odd and an even number of K blocks
    (MIXED, 192, 1088),
    (MIXED[::-1], 256, 1152),
    # up to 24
    ([7, 0, 33, 1, 64, 16, 5, 40] * 8, 192, 576),
    ([1, 24, 2, 65, 0, 9, 31, 32] * 8, 128, 640),
])
def test_several_units_a_pair(B, counts, H, I):
    """The first kernel's pairs do several units each, of tiles of all heights."""
    assert act_units(counts, I, 256) > 2 * PAIRS
    x, dy, W13, W2, bounds = expert_inputs(sum(counts) + I, counts, H, I, 3)
    for dt in (BF, F32):
        p = expert_problem(B, counts, H, I, 3, dx_dtype=dt, dw_dtype=dt)
        out = run_experts(B, p, x, dy, W13, W2, bounds, dx_sorted=empty(x.shape, dt), dW13=empty(W13.shape, dt),
                          dW2=empty(W2.shape, dt))
        check_experts(out, x, dy, W13, W2, bounds)


def test_more_units_a_pair_than_are_decoded_at_once(B):
    """Over 64 units a pair in both kernels, each with rows: the decoded units' two batches are used again."""
    E, H, I = 512, 64, 1280
    counts = [1 + e % 2 for e in range(E)]
    assert act_units(counts, I, 256) > 64 * PAIRS
    x, dy, W13, W2, bounds = expert_inputs(21, counts, H, I)

    def run(lo, hi):
        rows, n = slice(int(bounds[lo]), int(bounds[hi])), hi - lo
        p = expert_problem(B, counts[lo:hi], H, I)
        return run_experts(B, p, x[rows].clone(), dy[rows].clone(), W13[lo:hi], W2[lo:hi],
                           (bounds[lo:hi + 1] - bounds[lo]).astype(np.int32), dx_sorted=empty((rows.stop - rows.start, H)),
                           dW13=empty((n, 2 * I, H)), dW2=empty((n, H, I)))

    full = run(0, E)
    for lo in range(0, E, 32):          # a few units a pair each: the same bits, and in part against 64 bits
        part, hi = run(lo, lo + 32), lo + 32
        rows = slice(int(bounds[lo]), int(bounds[hi]))
        assert torch.equal(part["dx_sorted"], full["dx_sorted"][rows])
        assert torch.equal(part["dW13"], full["dW13"][lo:hi]) and torch.equal(part["dW2"], full["dW2"][lo:hi])
        if lo in (0, 256, 480):
            check_experts(part, x[rows], dy[rows], W13[lo:hi], W2[lo:hi], bounds[lo:hi + 1] - bounds[lo])


def test_experts_of_the_middle_of_a_batch(B):
    """Offsets that begin past the first row: rows before them do not count and are not written."""
    H, I, first = 192, 128, 37
    for counts in ([20, 0, 9], [200, 70, 300]):
        x, dy, W13, W2, bounds = expert_inputs(sum(counts), [first] + counts, H, I)
        x[:first], dy[:first] = float("nan"), float("nan")
        p = B.ExpertGradProblem.make(B.Problem.make(len(x), len(counts), 1, H, I))
        out = run_experts(B, p, x, dy, W13[1:], W2[1:], bounds[1:], dx_sorted=empty(x.shape), dW13=empty(W13[1:].shape),
                          dW2=empty(W2[1:].shape))
        assert (out["dx_sorted"][:first] == 7.0).all()
        out["dx_sorted"] = out["dx_sorted"][first:]
        check_experts(out, x[first:], dy[first:], W13[1:], W2[1:], bounds[1:] - first)


# ------------------------------------------------------------------ router, few slots

FORMS = [("softmax", True), ("sigmoid", True), ("sigmoid", False)]      # dl is zero but at the chosen experts


def check_few(got, x, w, logits, ids, dwt, score, renorm, size):
    """A term is off by `size` u; dx sums k terms, dw the slots of an expert, at most T * k."""
    dx, dw, dl, _ = got
    T, k = ids.shape
    want, mag = back.route(ref.f64(logits), ids, ref.f64(dwt), score, renorm)
    xx, ww = ref.f64(x), ref.f64(w)
    check(dl, want, size * U * mag, "dl")
    check(dx, want @ ww, (size + k + 1) * U * (mag @ np.abs(ww)), "dx")
    check(dw, want.T @ xx, (size + T * k + 1) * U * (mag.T @ np.abs(xx)), "dw")


@pytest.mark.parametrize("score,renorm", FORMS)
@pytest.mark.parametrize("T,E,k", [(128, 64, 8), (100, 12, 1), (250, 16, 1), (256, 300, 4), (37, 40, 6)])
def test_experts_of_many_slots(B, T, E, k, score, renorm):
    H = 320
    assert T * k <= min(1024, 16 * E)
    x, w, logits, ids, dwt = route_inputs(B, T + k, T, E, k, H, score, renorm)
    hot = ids.cpu().numpy().copy()
    hot[:, 0] = np.where(np.arange(T) % 3 == 0, E - 1, hot[:, 0])
    hot[T // 2] = -1
    assert np.bincount(hot[hot >= 0], minlength=E).max() >= 5
    p = B.RouterProblem.make(T, E, k, H, score=0 if score == "softmax" else 1, renormalize=renorm)
    got = run_route(B, p, x, w, logits, torch.from_numpy(hot).cuda(), dwt, dtype=F32)
    assert got[3] == 0
    check_few(got, x, w, logits, hot, dwt, score, renorm, 64)


@pytest.mark.parametrize("score,renorm", FORMS)
def test_experts_of_many_masked_slots(B, score, renorm):
    """Experts with five slots and more, some of them masked, repeated, far out or beside invalid ids."""
    T, E, k, H = 20, 12, 3, 128
    x, w, logits, _, dwt = route_inputs(B, 13, T, E, k, H, score, renorm)
    logits[0] = float("-inf")
    logits[1, 4] = float("-inf")
    logits[2, 4], logits[3, 4] = float("nan"), float("inf")
    logits[4] = -200.0                      # sigmoid scores underflow, their ratios do not
    logits[5] *= 20.0
    logits[6, 4], logits[6, 7] = -90.0, 90.0
    ids, _, _ = ref.route(ref.f64(logits), k, score, renorm)
    ids[1:12, 0] = 4
    ids[1:12, 1], ids[1:12, 2] = 7, 2
    ids[0] = [4, 7, 2]                      # a row with nothing left
    ids[8] = [4, 4, 7]                      # the same expert twice
    ids[9] = [4, -1, -1]
    ids[10] = [-1, 4, E]                    # an invalid id beside it
    ids[11] = [4, -5, 1 << 30]
    assert (ids == 4).sum() >= 12 and (ids == 7).sum() >= 5
    p = B.RouterProblem.make(T, E, k, H, score=0 if score == "softmax" else 1, renormalize=renorm)
    got = run_route(B, p, x, w, logits, torch.from_numpy(ids).cuda(), dwt, dtype=F32)
    assert got[3] == B.MOE_DEVERR_BAD_EXPERT_ID
    check_few(got, x, w, logits, ids, dwt, score, renorm, 300)      # arguments up to 200 in size


# ------------------------------------------------------------------ what is reported

@pytest.mark.parametrize("T,H,h", [(7, 7168, "bf16"), (16, 576, "fp32"), (300, 1088, "bf16"), (170, 12288, "bf16"),
                                   (900, 8192, "fp32")])
def test_norm_backward_reports_nothing(B, T, H, h):
    """Of the norm's workspace only the error word starts at zero, and it stays there."""
    dt = BF if h == "bf16" else F32
    g = gen(T)
    hh, dx, w = randn(g, (T, H), dt), randn(g, (T, H)), randn(g, (H,), BF, 0.1, 1.0)
    p = B.NormProblem.make(T, H, h_dtype=dt, eps=1e-5)
    ws = torch.full((B.moe_norm_backward_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    dh, dw = empty((T, H), dt), empty((H,))
    B.moe_norm_backward(p, hh, w, dx, dh, ws, dw=dw)
    assert B.moe_last_device_error(ws) == 0
    want, want_dw, mag, mag_dw = back.norm(ref.f64(hh), ref.f64(dx), ref.f64(w), 1e-5)
    check(dh, want, 90 * U * mag, "dh")
    check(dw, want_dw, (90 + T / 152 + 64) * U * mag_dw, "dw")


def test_step_reports_nothing_from_the_norm(B):
    T, E, k, H, I = 130, 16, 4, 256, 128
    s = Step(B, block_case(B, 3, T, E, k, H, I), T, E, k, H, I)
    s.forward()
    s.backward()
    assert s.errors() == [0, 0, 0, 0] and B.moe_last_device_error(s.norm_bws) == 0
