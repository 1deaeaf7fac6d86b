"""The router gradient's sums: over many tokens, and of infinite and largest logits' gradients."""
from __future__ import annotations

import torch
import pytest

import backward_reference as back
import block_reference as ref
from test_gpu_backward import B, BF, F32, U, check, gen, randn, route_inputs, run_route  # noqa: F401

pytestmark = pytest.mark.gpu

RANGE = 4096        # tokens of one unbroken sum on the tensor cores, at most


@pytest.mark.parametrize("T,E,H", [(262144, 128, 4096), (20000, 1024, 4928), (9000, 16, 64)])
def test_many_tokens_of_one_sign(B, T, E, H):
    """dw_router of same-signed terms, where truncated sums drift: within a bound that does not grow with the
    tokens but by the fp32 sum over their ranges."""
    g = gen(T)
    x, w = randn(g, (T, H)).abs_(), randn(g, (E, H), BF, H ** -0.5)
    logits, add = randn(g, (T, E), F32), torch.rand((T, E), generator=g, device="cuda") + 0.5
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    dwt = torch.zeros((T, 1), dtype=F32, device="cuda")
    p = B.RouterProblem.make(T, E, 1, H)
    _, dw, _, err = run_route(B, p, x, w, logits, ids, dwt, add, F32, wanted=("dw",))
    assert err == 0
    want = torch.zeros((E, H), dtype=torch.float64, device="cuda")
    for t in range(0, T, 16384):
        want += add[t:t + 16384].double().T @ x[t:t + 16384].double()
    off = ((dw.double() - want).abs() / want).max()
    assert off <= 2.0 ** -16 + back.mma_rel(2 * RANGE) + (T / RANGE + 77) * U, float(off)


def test_infinite_and_largest_gradients_of_logits(B):
    """An infinite gradient of a logit makes its products infinite, not NaN, and no other row's; one that a bf16
    leading part cannot hold stays finite."""
    T, E, k, H = 300, 40, 4, 192
    x, w, logits, ids, dwt = route_inputs(B, 8, T, E, k, H, "softmax", True)
    x *= 0.1
    assert (x[[7, 9, 11]] != 0).all() and (w[[2, 3, 5]] != 0).all()
    p = B.RouterProblem.make(T, E, k, H)
    add = torch.zeros((T, E), dtype=F32, device="cuda")
    clean = run_route(B, p, x, w, logits, ids, dwt, add, F32)
    inf, most = float("inf"), 3.4e38
    add[7, 3], add[9, 5], add[11, 2] = inf, -inf, most
    dx, dw, dl, err = run_route(B, p, x, w, logits, ids, dwt, add, F32)
    assert err == 0
    assert dl[7, 3] == inf and dl[9, 5] == -inf and dl[11, 2] == most
    for got, want in ((dx[7], inf * w[3].float()), (dx[9], -inf * w[5].float()), (dw[3], inf * x[7].float()),
                      (dw[5], -inf * x[9].float())):
        assert bool((got.float() == want).all())
    a, b = ref.f64(w[2]), ref.f64(x[11])
    check(dx[11], most * a, (2.0 ** -16 + back.mma_rel(128)) * most * abs(a), "dx")
    check(dw[2], most * b, (2.0 ** -16 + back.mma_rel(2 * T) + 152 * U) * most * abs(b), "dw")
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[[7, 9, 11]] = False
    cols = torch.ones(E, dtype=torch.bool, device="cuda")
    cols[[2, 3, 5]] = False
    assert torch.equal(dx[rows], clean[0][rows]) and torch.equal(dw[cols], clean[1][cols])
