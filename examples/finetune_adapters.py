#!/usr/bin/env python3
"""Trains the adapters of several requests at once beside one frozen INT8
projection, then serves single tokens with them.

Each of the tasks wants another low-rank change of the same projection; a
batch mixes their tokens with some that have no adapter.  Synthetic data, one
GPU, a few seconds:

  python examples/finetune_adapters.py [--steps 150] [--state-bits 8] [--bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w8a8_integer_linear_amd import AdaptedLinearW8A8  # noqa: E402


def train(steps=150, state_bits=32, bf16=False, tokens=1024, K=1024, N=768, tasks=3, rank=12,
          lr=3e-3, seed=0, say=print):
    """Returns (losses, layer, per-task relative error of single-token outputs)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape, std=1.0: torch.randn(shape, generator=g, device="cuda") * std  # noqa: E731
    weight = randn(N, K, std=K ** -0.5)
    # What each task adds to the projection, and adapters that start from nothing.
    wanted = [(randn(rank, K, std=K ** -0.5), randn(N, rank, std=0.3)) for _ in range(tasks)]
    adapters = [(randn(rank, K, std=K ** -0.5), torch.zeros(N, rank, device="cuda"), rank)
                for _ in range(tasks)]
    layer = AdaptedLinearW8A8(weight, torch.ones(K, device="cuda"), adapters,
                              dtype=torch.bfloat16 if bf16 else torch.float32, state_bits=state_bits)
    ids = (torch.arange(tokens, device="cuda") * (tasks + 1) // tokens - 1).to(torch.int32)

    def target(h, ids):
        n = h.float() * torch.rsqrt(h.float().square().mean(1, keepdim=True) + layer.eps)
        y = n @ weight.T
        for l, (A, B) in enumerate(wanted):
            y = torch.where((ids == l)[:, None], y + (n @ A.T) @ B.T, y)
        return y

    losses = []
    for step in range(1, steps + 1):
        x, res = (randn(tokens, K).to(torch.bfloat16) for _ in range(2))
        y, h = layer.forward(x, ids, residual=res)
        diff = y - target(h, ids)
        losses.append(diff.square().mean().item())
        layer.backward((diff * (2.0 / N)).to(torch.bfloat16))
        layer.adamw_step(lr, seed=7, step=step)
        if step == 1 or step % 50 == 0:
            say(f"step {step:4d}  loss {losses[-1]:.5f}")
    # Serving: one token per request, every adapter in the same call.
    ids = torch.arange(-1, tasks, device="cuda", dtype=torch.int32)
    x = randn(tasks + 1, K).to(torch.bfloat16)
    y, h = layer.forward(x, ids, save=False)
    want = target(h, ids)
    error = ((y - want).norm(dim=1) / want.norm(dim=1)).tolist()
    say("single tokens, relative error (no adapter first): " + " ".join(f"{e:.3f}" for e in error))
    return losses, layer, error


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=150)
    ap.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    ap.add_argument("--bf16", action="store_true", help="adapters in bf16, rounded stochastically")
    a = ap.parse_args()
    train(a.steps, a.state_bits, a.bf16)


if __name__ == "__main__":
    main()
