"""The training example runs, and a micro-batch's gradients are those of torch's
differentiation in 64 bits."""
from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    from moe_routed_expert_routing_gb300.build import build
    build()
    spec = importlib.util.spec_from_file_location("moe_block_training", os.path.join(ROOT, "examples", "moe_block_training.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def test_example_runs():
    _, losses = load().main(["--tokens", "96", "--steps", "3", "--shape", "8,2,256,128"])
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


def test_gradients_of_two_micro_batches():
    """Rows go through bf16 some five times on the way (x, the block's output and stream, y's and x's gradients, the
    experts' inner rows), 2^-8 each at most and independent: 2 * 2^-8 of a result's norm, where uniform
    roundings come to a quarter of that."""
    example = load()
    T, E, k, H, I = 70, 8, 2, 256, 128
    block = example.Block(T, E, k, H, I, seed=3)
    block.capture()
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    leaf = {n: w.double().cpu().requires_grad_() for n, w in block.weights.items()}
    for _ in range(2):
        block.h.copy_(torch.randn((T, H), generator=g, device="cuda"))
        block.target.copy_(torch.randn((T, H), generator=g, device="cuda"))
        block.graph.replay()
        h, target, ids = block.h.double().cpu(), block.target.double().cpu(), block.ids.cpu().long()
        x = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * leaf["w_pre"]
        p = torch.softmax(x @ leaf["w_router"].T, 1).gather(1, ids)
        p = p / p.sum(1, keepdim=True)
        y = torch.zeros_like(h)
        for e in range(E):
            t, j = (ids == e).nonzero(as_tuple=True)
            gu = x[t] @ leaf["W13"][e].T
            y = y.index_add(0, t, p[t, j, None] * ((torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ leaf["W2"][e].T))
        loss = ((h + y - target) ** 2).mean() / 2
        loss.backward()
        assert abs(float(block.loss) - float(loss.detach())) <= 2 ** -8 * float(loss.detach())
    block.check()
    for n, w in leaf.items():
        got = block.grads[n].double().cpu()
        off = float((got - w.grad).norm() / w.grad.norm())
        assert off <= 2 * 2.0 ** -8, (n, off)
