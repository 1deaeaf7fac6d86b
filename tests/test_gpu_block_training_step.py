"""The training example's update of the weights from its gradients."""
from __future__ import annotations

import pytest
import torch

from test_gpu_block_training_example import load

pytestmark = pytest.mark.gpu


def test_a_step_is_gradient_descent_on_the_mean():
    """w - lr g / n in fp32, rounded once to bf16, for the gradients of two micro-batches; they start at zero again."""
    T, E, k, H, I = 70, 8, 2, 256, 128
    block = load().Block(T, E, k, H, I, seed=5)
    block.capture()
    assert all(not g.any() for g in block.grads.values())
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    for _ in range(2):
        block.h.copy_(torch.randn((T, H), generator=g, device="cuda"))
        block.target.copy_(torch.randn((T, H), generator=g, device="cuda"))
        block.graph.replay()
    old = {n: w.clone() for n, w in block.weights.items()}
    grads = {n: v.clone() for n, v in block.grads.items()}
    assert all(v.any() for v in grads.values())
    block.step(16.0, 2)
    block.check()
    for n, w in block.weights.items():
        want = (old[n].double() - grads[n].double() * 8.0).to(torch.float32)
        # half a step of bf16 for the rounding; the product and the difference in fp32 add a 2^-23 of their size
        size = old[n].double().abs() + grads[n].double().abs() * 8.0
        assert ((w.double() - want.double()).abs() <= 2.0 ** -8 * want.double().abs() + 2.0 ** -22 * size).all(), n
        assert not torch.equal(w, old[n]) and not block.grads[n].any(), n
