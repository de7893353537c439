"""A training step of one expert block, every heavy operator from the library:

  h0 = table[tokens]
  h1 = h0 + experts(layer_norm(h0))        router: layer_norm(h0) Wr, top-k
  loss = cross entropy of layer_norm(h1) against the output weights

then the backward pass, the gradients' global norm clipped, and plain SGD.
PyTorch does what is small here: the embedding lookup, the router's matrix,
residual sums and the update.

  python examples/train_step.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from mixture_experts_layer_18_gb300.layer import MoELayer  # noqa: E402
from mixture_experts_layer_18_gb300.training import CrossEntropy, GradClip, LayerNorm  # noqa: E402


class Block:
    """Weights, gradients and buffers of the block for T tokens."""

    def __init__(self, T=2048, H=512, E=16, I=256, top_k=2, V=5003, ignore_index=-100, seed=0):
        self.T, self.H, self.V = T, H, V
        g = torch.Generator(device="cuda").manual_seed(seed)

        def bf16(*shape, scale):
            return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()
        ones, zeros = (torch.full((H,), v, device="cuda") for v in (1.0, 0.0))
        self.w = dict(
            table=bf16(V, H, scale=1.0), gamma1=ones.clone(), beta1=zeros.clone(),
            Wr=torch.randn((H, E), generator=g, device="cuda") / H ** 0.5,
            W13=bf16(E, H, 2 * I, scale=H ** -0.5), W2=bf16(E, I, H, scale=I ** -0.5),
            gamma2=ones.clone(), beta2=zeros.clone(), Wout=bf16(V, H, scale=H ** -0.5))
        self.g = {k: torch.zeros_like(v) for k, v in self.w.items()}
        bf, f32 = torch.bfloat16, torch.float32
        self.norm1 = LayerNorm(T, H, dtype=bf, weight_dtype=f32)
        self.norm2 = LayerNorm(T, H, dtype=bf, weight_dtype=f32)
        self.moe = MoELayer(T, H, E, I, top_k, mode="bf16")
        self.xent = CrossEntropy(T, H, V, ignore_index=ignore_index)
        self.clip = GradClip(self.g.values())
        self.one = torch.ones(1, device="cuda")
        b = dict(dtype=bf, device="cuda")
        self.n1, self.n2, self.y, self.dn2, self.dh1, self.dn1, self.dh0 = (
            torch.empty((T, H), **b) for _ in range(7))
        self.dgate = torch.empty((T, top_k), device="cuda")
        self.dlogits = torch.empty((T, E), device="cuda")

    def forward(self, tokens, targets):
        w = self.w
        self.h0 = w["table"][tokens]
        self.norm1.forward(self.h0, w["gamma1"], w["beta1"], self.n1)
        self.moe.route(self.n1.float() @ w["Wr"])
        self.moe.forward(self.n1, w["W13"], w["W2"], self.y)
        self.h1 = self.h0 + self.y
        self.norm2.forward(self.h1, w["gamma2"], w["beta2"], self.n2)
        self.xent.forward(self.n2, w["Wout"], targets)
        return self.xent.mean

    def backward(self, tokens, targets):
        w, g = self.w, self.g
        self.xent.backward(self.n2, w["Wout"], targets, self.one, self.dn2, g["Wout"], reduction="mean")
        self.norm2.backward(self.dn2, self.h1, w["gamma2"], self.dh1, g["gamma2"], g["beta2"])
        self.moe.backward(self.dh1, w["W13"], w["W2"], self.dn1, g["W13"], g["W2"], self.dgate)
        self.moe.route_backward(self.dgate, self.dlogits)
        torch.mm(self.n1.float().T, self.dlogits, out=g["Wr"])
        self.dn1 += (self.dlogits @ w["Wr"].T).to(self.dn1.dtype)
        self.norm1.backward(self.dn1, self.h0, w["gamma1"], self.dh0, g["gamma1"], g["beta1"])
        self.dh0 += self.dh1
        g["table"].zero_()
        g["table"].index_put_((tokens,), self.dh0, accumulate=True)

    def step(self, tokens, targets, lr, max_norm):
        """One step; returns the loss before it and the gradients' norm (device numbers)."""
        loss = self.forward(tokens, targets).clone()
        self.backward(tokens, targets)
        self.clip.clip(max_norm)
        for k, v in self.w.items():
            v -= (lr * self.g[k].float()).to(v.dtype)
        return loss, self.clip.norm


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=2.0)
    ap.add_argument("--max-norm", type=float, default=1.0)
    a = ap.parse_args()
    block = Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    # a task that one block can learn: the next token is a fixed function of the token
    table = torch.randperm(block.V, generator=g, device="cuda")
    for i in range(a.steps):
        tokens = torch.randint(0, 64, (block.T,), generator=g, device="cuda")
        targets = table[tokens]
        targets[torch.rand(block.T, generator=g, device="cuda") < 0.1] = -100      # prompt tokens
        loss, norm = block.step(tokens, targets, a.lr, a.max_norm)
        print(f"step {i:3d}  loss {float(loss):.4f}  gradient norm {float(norm):.3f}")
    if any(op.device_status() for op in (block.moe, block.xent, block.clip)):
        raise SystemExit("a device error was reported")


if __name__ == "__main__":
    main()
