"""Training steps of one mixture-of-experts block.

Each step goes forward through the operators (moe_norm, moe_route, moe_dispatch,
moe_expert_compute, moe_combine and the residual sum) and back through their
gradients, for several micro-batches whose expert gradients add up in fp32, then
takes a step of plain gradient descent on the weights. A micro-batch is one CUDA
graph, forward and backward. The loss is the mean square distance of the block's
stream to a target.

    python examples/moe_block_training.py [--tokens 512] [--micro 2] [--steps 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_routed_expert_routing_gb300 import binding as B  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Block:
    """Weights, their gradients, and the buffers of one micro-batch of T tokens."""

    def __init__(self, T, E, k, H, I, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape, std=1.0, mean=0.0):
            return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(BF16)

        def new(*shape, dtype=BF16):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        def ws(n):
            return new(n, dtype=torch.uint8)

        self.weights = {"w_pre": randn(H, std=0.1, mean=1.0), "w_router": randn(E, H, std=H ** -0.5),
                        "W13": randn(E, 2 * I, H, std=H ** -0.5), "W2": randn(E, H, I, std=I ** -0.5)}
        self.experts, self.router, self.norm = B.Problem.make(T, E, k, H, I), B.RouterProblem.make(T, E, k, H), B.NormProblem.make(T, H)
        # expert gradients in fp32, added to what the micro-batches before left
        self.expert_grad = B.ExpertGradProblem.make(self.experts, dw_dtype=F32, accumulate=True)
        self.grads = {"W13": new(E, 2 * I, H, dtype=F32), "W2": new(E, H, I, dtype=F32),
                      "w_router": new(E, H, dtype=F32), "w_pre": new(H, dtype=F32)}
        self.bufs = B.Buffers(self.experts)
        self.h, self.target, self.out, self.dout, self.dh = (new(T, H) for _ in range(5))
        self.x, self.dx, self.dy, self.dx_sorted = new(T, H), new(T, H), new(T * k, H), new(T * k, H)
        self.ids, self.topk, self.dtopk = new(T, k, dtype=torch.int32), new(T, k, dtype=F32), new(T, k, dtype=F32)
        self.logits, self.dw_router, self.dw_pre = new(T, E, dtype=F32), new(E, H, dtype=F32), new(H)
        self.loss = new(1, dtype=F32)
        self.route_ws = ws(B.moe_route_workspace_size(self.router))
        self.route_grad_ws = ws(B.moe_route_backward_workspace_size(self.router))
        self.expert_grad_ws = ws(B.moe_expert_backward_workspace_size(self.expert_grad))
        self.norm_grad_ws = ws(B.moe_norm_backward_workspace_size(self.norm))

    def forward(self):
        w, b = self.weights, self.bufs
        B.moe_norm(self.norm, self.h, w["w_pre"], self.x)
        B.moe_route(self.router, self.x, w["w_router"], self.ids, self.topk, self.route_ws, logits=self.logits)
        B.moe_dispatch(self.experts, self.ids, b.expert_offsets, b.perm, b.inv, b.ws, x=self.x, x_sorted=b.x_sorted)
        B.moe_expert_compute(self.experts, b.x_sorted, b.expert_offsets, w["W13"], w["W2"], b.y_sorted, b.ws)
        B.moe_combine(self.experts, b.y_sorted, b.inv, self.topk, b.out)
        torch.add(self.h, b.out, out=self.out)

    def backward(self):
        """Gradients of mean((out - target)^2) / 2: into dh, and added to self.grads."""
        w, b = self.weights, self.bufs
        diff = self.out.float() - self.target.float()
        self.loss.copy_((diff * diff).mean() / 2)
        self.dout.copy_(diff / diff.numel())
        B.moe_combine_backward(self.experts, self.dout, b.inv, self.topk, self.dy, y_sorted=b.y_sorted, d_weights=self.dtopk)
        B.moe_expert_backward(self.expert_grad, b.x_sorted, b.expert_offsets, w["W13"], w["W2"], self.dy,
                              self.expert_grad_ws, dx_sorted=self.dx_sorted, dW13=self.grads["W13"], dW2=self.grads["W2"])
        B.moe_route_backward(self.router, self.x, w["w_router"], self.logits, self.ids, self.dtopk, self.route_grad_ws,
                             dx=self.dx, dw_router=self.dw_router)
        # the experts' part of x's gradient on top of the router's, then through the norm onto the stream's own
        B.moe_dispatch_backward(self.experts, self.dx_sorted, b.inv, self.dx, dx_add=self.dx)
        B.moe_norm_backward(self.norm, self.h, w["w_pre"], self.dx, self.dh, self.norm_grad_ws, dh_add=self.dout, dw=self.dw_pre)
        self.grads["w_router"] += self.dw_router
        self.grads["w_pre"] += self.dw_pre

    def capture(self):
        """One micro-batch, forward and backward, as a graph (inputs: self.h and self.target)."""
        self.forward()
        self.backward()          # the first calls on a device stay outside capture
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.forward()
            self.backward()
        for g in self.grads.values():
            g.zero_()

    def step(self, lr, n_micro):
        for n, w in self.weights.items():
            w.copy_(w.float() - self.grads[n] * (lr / n_micro))
            self.grads[n].zero_()

    def check(self):
        for name, ws in (("route", self.route_ws), ("experts", self.bufs.ws), ("route backward", self.route_grad_ws),
                         ("experts backward", self.expert_grad_ws), ("norm backward", self.norm_grad_ws)):
            if B.moe_last_device_error(ws):
                raise RuntimeError(f"device error in {name}")


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--micro", type=int, default=2)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--lr", type=float, default=20.0)
    ap.add_argument("--shape", default="32,4,1024,512", help="E,k,H,I")
    args = ap.parse_args(argv)
    E, k, H, I = map(int, args.shape.split(","))
    block = Block(args.tokens, E, k, H, I)
    block.capture()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    batches = [(torch.randn((args.tokens, H), generator=g, device="cuda").to(BF16),
                torch.randn((args.tokens, H), generator=g, device="cuda").to(BF16)) for _ in range(args.micro)]
    losses, start, end = [], torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(args.steps):
        loss = torch.zeros(1, device="cuda")
        for h, target in batches:
            block.h.copy_(h)
            block.target.copy_(target)
            block.graph.replay()
            loss += block.loss / args.micro
        block.step(args.lr, args.micro)
        losses.append(loss)
    end.record()
    torch.cuda.synchronize()
    block.check()
    losses = [float(v) for v in losses]
    print(f"E={E} k={k} H={H} I={I}, {args.micro} x {args.tokens} tokens a step: loss {losses[0]:.4f} -> {losses[-1]:.4f} in "
          f"{args.steps} steps, {start.elapsed_time(end) / args.steps:.2f} ms a step")
    return block, losses


if __name__ == "__main__":
    main()
