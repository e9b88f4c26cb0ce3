"""A residual stack of gated feed-forward layers in 8 bits: decoding, and tuning its norms and
gates through the frozen weights.

    python examples/feed_forward.py [--layers 4] [--width 4096] [--hidden 14336] [--tokens 1024]

One layer, all of it in the library's kernels:

    r, (q, s) = block_norm(r, y)      finished block's norm and gate, residual, next norm, int8
    h = gated_i8(q, s)                both projections, activation and product
    y = linear_i8(quantize(h))        back to the width of the stream

The backward pass walks the layers in reverse with the operators' own backward functions.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_weight_only_offline_amd as Q  # noqa: E402


class FeedForwardStack:
    """Random int8 weights; norm weights and gates in float32 (`params`), which can be tuned."""

    def __init__(self, layers: int, width: int, hidden: int, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(n, k):
            return Q.quantize_activations((torch.randn((n, k), generator=g, device=device) / k ** 0.5).bfloat16())
        self.up_gate = [Q.pack_gated(*weight(hidden, width), *weight(hidden, width)) for _ in range(layers)]
        self.down = [Q.pack_channel(*weight(width, hidden)) for _ in range(layers)]

        def ones(value=1.0):
            return torch.full((width,), value, device=device)
        # pre[i] is the norm before layer i, pre[layers] the one before the output
        self.params = {"pre": [ones() for _ in range(layers + 1)], "post": [ones() for _ in range(layers)],
                       "gate": [ones(0.5) for _ in range(layers)]}

    def _norm_args(self, i):
        """block_norm's parameters after layer i - 1 (i = 0: before the first layer)."""
        p = self.params
        if i == 0:
            return {"pre_weight": p["pre"][0]}
        return {"pre_weight": p["pre"][i], "post_weight": p["post"][i - 1], "gate": p["gate"][i - 1]}

    def forward(self, x: torch.Tensor, keep: bool = False):
        """bf16 output for the float32 stream x [tokens, width]; keep: also what backward() reads."""
        n = len(self.down)
        r, y, saved = x, None, []
        for i in range(n + 1):
            r, out = Q.block_norm(r, y, int8=i < n, **self._norm_args(i))
            if i == n:
                saved.append((r, y, None))
                break
            h, raw = Q.gated_i8(*out, self.up_gate[i], keep_raw=True) if keep else (Q.gated_i8(*out, self.up_gate[i]), None)
            if keep:
                saved.append((r, y, raw))
            y = Q.linear_i8(*Q.quantize_activations(h), self.down[i])
        return (out, saved) if keep else out

    def backward(self, dx: torch.Tensor, saved):
        """Gradients of `params` and of the input for dx, the gradient of the output."""
        n = len(self.down)
        grads = {k: [None] * len(v) for k, v in self.params.items()}
        dr = None
        for i in range(n, -1, -1):
            r, y, _ = saved[i]
            dr, dy, dpost, dpre, dgate = Q.block_norm_backward(dx, dr, r, y, **self._norm_args(i))
            grads["pre"][i] = dpre
            if i == 0:
                return grads, dr
            grads["post"][i - 1], grads["gate"][i - 1] = dpost, dgate
            dh = Q.linear_i8_backward(dy, self.down[i - 1])
            dx, _ = Q.gated_i8_backward(dh, saved[i - 1][2], self.up_gate[i - 1])

    def tune(self, x: torch.Tensor, target: torch.Tensor, rate: float) -> torch.Tensor:
        """One step of gradient descent on half the mean squared distance to target; its value
        before the step."""
        out, saved = self.forward(x, keep=True)
        off = out.float() - target
        grads, _ = self.backward((off / out.shape[0]).bfloat16(), saved)
        for name, tensors in self.params.items():
            for p, g in zip(tensors, grads[name]):
                p.sub_(rate * g)
        return 0.5 * off.square().sum() / out.shape[0]


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--layers", type=int, default=4)
    a.add_argument("--width", type=int, default=4096)
    a.add_argument("--hidden", type=int, default=14336)
    a.add_argument("--tokens", type=int, default=1024)
    a.add_argument("--steps", type=int, default=8)
    a = a.parse_args()
    stack = FeedForwardStack(a.layers, a.width, a.hidden)

    def timed(f, n):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n

    token = torch.randn((1, a.width), device="cuda")
    print(f"one token through {a.layers} layers: {timed(lambda: stack.forward(token), 50) * 1e6:.1f} us", flush=True)
    x = torch.randn((a.tokens, a.width), device="cuda")
    print(f"{a.tokens} tokens, forward: {timed(lambda: stack.forward(x), 10) * 1e3:.2f} ms", flush=True)
    target = stack.forward(x).float() + 0.1 * torch.randn((a.width,), device="cuda") * torch.randn_like(x)
    for name in ("post", "gate"):
        for p in stack.params[name]:
            p.mul_(1 + 0.2 * torch.randn_like(p))
    for i in range(a.steps):
        print(f"step {i}: loss {float(stack.tune(x, target, rate=0.2)):.4f}", flush=True)


if __name__ == "__main__":
    main()
