"""A stack of mixture-of-experts blocks: a prompt, then decoded tokens.

Each block norms the residual stream, routes, runs the routed experts and goes
back into the stream through a norm and a residual scale. The prompt takes the
operators one by one (moe_norm, moe_route, moe_forward, moe_norm_residual, which
also norms for the next block); the decoded tokens take moe_layer, all blocks of
a step in one CUDA graph that is replayed with the step's token count on the
device. What stands between the blocks of a language model (attention) is left
out, and the "next token" is the stream's own row, so this shows the calls and
times them, nothing else.

    python examples/moe_block.py [--blocks 4] [--prompt 512] [--batch 8] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_routed_expert_routing_gb300 import binding as B  # noqa: E402


class Block:
    """One block's weights, drawn at random at the scale of trained ones."""

    def __init__(self, g, E, H, I):
        def randn(*shape, std=1.0, mean=0.0):
            return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(mean, std, generator=g)

        self.w_pre, self.w_post = randn(H, std=0.1, mean=1.0), randn(H, std=0.1, mean=1.0)
        self.w_router = randn(E, H, std=H ** -0.5)
        self.W13, self.W2 = randn(E, 2 * I, H, std=H ** -0.5), randn(E, H, I, std=I ** -0.5)


class Stack:
    def __init__(self, blocks, E, k, H, I, scale=0.5, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.E, self.k, self.H, self.I, self.scale = E, k, H, I, scale
        self.blocks = [Block(g, E, H, I) for _ in range(blocks)]
        self.w_final = torch.ones(H, dtype=torch.bfloat16, device="cuda")

    def problems(self, T):
        return (B.Problem.make(T, self.E, self.k, self.H, self.I),
                B.RouterProblem.make(T, self.E, self.k, self.H),
                B.NormProblem.make(T, self.H, norm_block=True, residual_scale=self.scale))

    def prompt(self, h):
        """All rows of h through the blocks, in place; returns the final norm of the rows."""
        T = h.shape[0]
        experts, router, norm = self.problems(T)
        bufs = B.Buffers(experts)
        ids = torch.empty((T, self.k), dtype=torch.int32, device="cuda")
        weights = torch.empty((T, self.k), device="cuda")
        ws = torch.zeros(B.moe_route_workspace_size(router), dtype=torch.uint8, device="cuda")
        x = torch.empty_like(h)
        B.moe_norm(norm, h, self.blocks[0].w_pre, x)
        for i, b in enumerate(self.blocks):
            w_next = self.blocks[i + 1].w_pre if i + 1 < len(self.blocks) else self.w_final
            B.moe_route(router, x, b.w_router, ids, weights, ws)
            B.moe_forward(experts, x, ids, weights, b.W13, b.W2, bufs.expert_offsets, bufs.perm, bufs.out, bufs.ws)
            B.moe_norm_residual(norm, h, bufs.out, h, w_post=b.w_post, w_next=w_next, x_next=x)
        for name, w in (("route", ws), ("forward", bufs.ws)):
            if B.moe_last_device_error(w):
                raise RuntimeError(f"device error in {name}")
        return x


class Decoder:
    """Decode steps of up to `batch` tokens: every block of a step in one graph."""

    def __init__(self, stack, batch):
        experts, router, norm = stack.problems(batch)
        self.h = torch.zeros((batch, stack.H), dtype=torch.bfloat16, device="cuda")
        self.x = torch.zeros_like(self.h)
        self.tokens = torch.zeros(1, dtype=torch.int32, device="cuda")
        layer = B.LayerProblem.make(experts, router, norm)
        self.ws = torch.zeros(B.moe_layer_workspace_size(layer), dtype=torch.uint8, device="cuda")
        ids = torch.empty((batch, stack.k), dtype=torch.int32, device="cuda")
        weights = torch.empty((batch, stack.k), device="cuda")
        offsets = torch.empty(stack.E + 1, dtype=torch.int32, device="cuda")
        perm = torch.empty(batch * stack.k, dtype=torch.int32, device="cuda")

        def step():
            for i, b in enumerate(stack.blocks):
                last = i + 1 == len(stack.blocks)
                B.moe_layer(layer, self.h, b.w_pre, b.w_router, b.W13, b.W2, ids, weights, offsets, perm, self.h, self.ws,
                            w_post=b.w_post, w_next=stack.w_final if last else None, x_next=self.x if last else None,
                            d_num_tokens=self.tokens)

        step()                                   # the first call on a device stays outside capture
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            step()

    def run(self, rows):
        """One step for rows[T, H] (T <= batch): the blocks' output and its final norm, as views."""
        T = rows.shape[0]
        self.h[:T].copy_(rows)
        self.tokens.fill_(T)
        self.graph.replay()
        return self.h[:T], self.x[:T]


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--blocks", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--shape", default="64,4,1024,512", help="E,k,H,I")
    args = ap.parse_args(argv)
    E, k, H, I = map(int, args.shape.split(","))
    stack = Stack(args.blocks, E, k, H, I)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    prompt = torch.randn((args.prompt, H), generator=g, device="cuda").bfloat16()
    h = prompt.clone()
    x = stack.prompt(h)
    decoder = Decoder(stack, args.batch)
    # the prompt's last rows through the decoder give the same stream, up to bf16 roundings
    n = min(args.batch, args.prompt)
    h_dec, x_dec = decoder.run(prompt[-n:])
    diff = ((h_dec.float() - h[-n:].float()).norm() / h[-n:].float().norm()).item()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    row = x_dec.clone()
    start.record()
    for _ in range(args.steps):
        _, x_dec = decoder.run(row)
        row.copy_(x_dec)
    end.record()
    torch.cuda.synchronize()
    if B.moe_last_device_error(decoder.ws):
        raise RuntimeError("device error in the decoder")
    us = start.elapsed_time(end) * 1e3 / args.steps
    print(f"{args.blocks} blocks E={E} k={k} H={H} I={I}: prompt of {args.prompt} rows, then {args.steps} steps of "
          f"{n} tokens, {us:.1f} us a step; decoder against prompt {diff:.2e}")
    return diff, bool(torch.isfinite(x).all()) and bool(torch.isfinite(row).all())


if __name__ == "__main__":
    main()
