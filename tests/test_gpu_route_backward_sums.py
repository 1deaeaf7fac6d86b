"""The router gradient's sums over many tokens."""
from __future__ import annotations

import torch
import pytest

import backward_reference as back
from test_gpu_backward import B, BF, F32, U, gen, randn, run_route  # noqa: F401

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
