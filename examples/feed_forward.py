"""A gated feed-forward block trained in bf16, then served in 8 bits.

A block is fitted to another one's outputs on random inputs: each step runs
some microbatches forward and backward (``GatedFeedForwardPlan``), their weight
gradients added up in fp32, and takes one step of gradient descent on fp32
copies of the weights.  Then the weights are brought to e4m3 with a scale for
each block of 128 x 128 (``quantize_blocks``), and single tokens and whole
prompts are answered with them (``ScaledFeedForwardPlan``).

    python examples/feed_forward.py [--width 512] [--hidden 1408] [--tokens 300] [--steps 5]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fusion_b2b_gemm_gb300 as b2b  # noqa: E402


def normal(g, rows, cols):
    """A weight of unit gain."""
    return torch.randn(rows, cols, generator=g, device="cuda") / rows ** 0.5


def gradients(plan, weights, x, target, microbatches):
    """Gradients of the mean squared error over all of x, added up over microbatches in fp32, and the error."""
    total = tuple(torch.zeros(w.shape, dtype=torch.float32, device="cuda") for w in weights)
    error = 0.0
    for part, want in zip(x.chunk(microbatches), target.chunk(microbatches)):
        y, kept = plan.forward(part, *weights)
        off = y.float() - want.float()
        error = error + off.square().sum() / target.numel()
        dy = (off * (2 * x.shape[0] / target.numel())).bfloat16()  # (over the tokens below, in fp32)
        plan.backward(dy, part, *weights, kept, input_grad=False, weight_grads=total)
    return tuple(t / x.shape[0] for t in total), error


def train(width, hidden, tokens, steps, microbatches=3, rate=0.5, seed=0):
    """Weights after `steps` steps, and the error before each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes = (width, hidden), (width, hidden), (hidden, width)
    teacher = [normal(g, *s).bfloat16() for s in shapes]
    masters = [normal(g, *s) for s in shapes]
    plan = b2b.GatedFeedForwardPlan("bf16", width, hidden)
    errors = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
        grads, error = gradients(plan, [m.bfloat16() for m in masters], x, plan.run(x, *teacher), microbatches)
        errors.append(float(error))
        for m, d in zip(masters, grads):
            m -= rate * d
    if plan.status():
        raise RuntimeError(f"device status {plan.status()}")
    return [m.bfloat16() for m in masters], errors


def serve(weights, x):
    """The block's outputs on e4m3 weights."""
    width, hidden = weights[0].shape
    plan = b2b.ScaledFeedForwardPlan("bf16", width, hidden)
    eight = [t for w in weights for t in b2b.quantize_blocks(w.t().contiguous(), 128)]
    y = plan.run(x, *eight)
    if plan.status():
        raise RuntimeError(f"device status {plan.status()}")
    return y


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("width", 512), ("hidden", 1408), ("tokens", 300), ("steps", 5)):
        p.add_argument(f"--{name}", type=int, default=default)
    a = p.parse_args()
    weights, errors = train(a.width, a.hidden, a.tokens, a.steps)
    print("error before each step:", " ".join(f"{e:.4f}" for e in errors))
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    exact = b2b.GatedFeedForwardPlan("bf16", a.width, a.hidden).run(x, *weights).float()
    for rows in (1, a.tokens):
        y = serve(weights, x[:rows]).float()
        off = ((y - exact[:rows]).norm() / exact[:rows].norm()).item()
        print(f"{rows} tokens in 8 bits: {100 * off:.1f} % off the 16-bit block")


if __name__ == "__main__":
    main()
