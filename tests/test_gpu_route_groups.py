"""moe_route's limited groups whose value is the sum of two keys, for more
tokens than the few-token kernels take: groups of every width, group counts that
do not divide a warp, and biases of -inf that leave a group one expert or none."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_reference as ref
from test_gpu_block import B, check, gen, grid_inputs, randn, run_route  # noqa: F401  (B is the module's fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value encountered in subtract")]

CASES = [
    # T, E, k, H, score, groups, keep
    (193, 256, 8, 512, "sigmoid", 8, 4),
    (700, 256, 8, 256, "softmax", 8, 3),
    (193, 1024, 16, 128, "sigmoid", 32, 5),
    (700, 64, 6, 192, "sigmoid", 32, 9),        # two experts a group
    (257, 160, 6, 128, "sigmoid", 10, 4),       # three lanes a group, two left over
    (700, 70, 4, 64, "softmax", 10, 1),
    (193, 51, 3, 64, "sigmoid", 17, 2),         # one lane a group
    (300, 384, 8, 256, "sigmoid", 2, 1),
    (1500, 512, 40, 64, "sigmoid", 4, 2),       # more experts than one warp-wide list holds
]


def run(B, T, E, k, H, score, groups, keep, bias, seed):
    x, w = grid_inputs(gen(seed), T, E, H)
    p = B.RouterProblem.make(T, E, k, H, score=int(score == "sigmoid"), n_group=groups, topk_group=keep, group_top=2,
                             scale=2.5)
    ids, wt, ws = run_route(B, p, x, w, bias=bias)
    want_ids, want_w, margin = ref.route(ref.f64(x) @ ref.f64(w).T, k, score, True, ref.f64(bias), groups, keep, 2, 2.5)
    sure = margin > 2e-6              # keys are fp32 sums of a score and a bias
    assert sure.mean() > 0.5
    got = ids.cpu().numpy()
    assert np.array_equal(got[sure], want_ids[sure])
    check(wt[torch.from_numpy(sure).cuda()], want_w[sure], np.abs(want_w[sure]) * 1e-5 + 1e-37, "weights")
    assert B.moe_last_device_error(ws) == 0
    return got, wt


@pytest.mark.parametrize("T,E,k,H,score,groups,keep", CASES)
def test_two_best_of_a_group(B, T, E, k, H, score, groups, keep):
    run(B, T, E, k, H, score, groups, keep, randn(gen(E + groups), (E,), torch.float32, 0.1), T + E)


@pytest.mark.parametrize("T", [7, 193, 700])
@pytest.mark.parametrize("E,groups,keep,k", [(64, 8, 3, 6), (160, 10, 4, 9), (96, 32, 8, 5)])
def test_groups_of_one_eligible_expert_or_none(B, T, E, groups, keep, k):
    """A group with fewer than two eligible experts has the value -inf: it stays only where too few others are left,
    and then its one expert may be chosen."""
    size = E // groups
    for whole in (groups - 1, keep, keep - 1, 0):         # groups with all their experts; the next has one, the rest none
        bias = randn(gen(E + whole), (E,), torch.float32, 0.1)
        bias[whole * size:] = float("-inf")
        if whole < groups:
            bias[whole * size + size - 1] = 0.05
        got, wt = run(B, T, E, k, 128, "sigmoid", groups, keep, bias, T + whole)
        eligible = min(whole, keep) * size + (1 if whole < keep else 0)
        assert ((got >= 0).sum(1) == min(k, eligible)).all()
        assert (wt[torch.from_numpy(got < 0).cuda()] == 0).all()
