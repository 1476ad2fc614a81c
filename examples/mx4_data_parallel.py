"""Data-parallel training of one 4-bit linear layer over R virtual ranks.

Every rank runs y = residual + dropout(x W^T) and its backward pass on its own
micro-batch with both products and their gradients in microscaled 4 bits; the
weight gradients are rounded stochastically to 4 bits and summed by the ring
AllReduce on that wire; every rank takes the same step.  No dropout mask, no
dropped-out gradient and no random number is ever stored: each is computed
again from (seed, subsequence, element) where it is needed.

    python examples/mx4_data_parallel.py [--ranks 4] [--tokens 512] [--features 1024] [--steps 30]

Prints the loss of a fixed linear target, first with a binary32 ring AllReduce
of the same gradients for comparison, then on the 4-bit wire.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_allreduce_reducescatter_gb300 as rr  # noqa: E402

SEED = 2024


def subsequence(step: int, rank: int, use: int) -> int:
    """One subsequence of the generator for each step, rank and use."""
    return (step * 64 + rank) * 4 + use


def train(ranks: int, tokens: int, features: int, steps: int, four_bits: bool, p: float = 0.1):
    g = torch.Generator(device="cuda").manual_seed(1)
    target = torch.randn((features, features), generator=g, device="cuda") / features ** 0.5
    weights = [torch.zeros((features, features), dtype=torch.bfloat16, device="cuda") for _ in range(ranks)]
    losses = []
    for step in range(steps):
        grads, loss = [], 0.0
        for r in range(ranks):
            x = torch.randn((tokens, features), generator=g, device="cuda").to(torch.bfloat16)
            want = x + (x.float() @ target.t()).to(torch.bfloat16)
            w = weights[r].detach().requires_grad_()
            drop = rr.Dropout(p, SEED, subsequence(step, r, 0))
            y = rr.mx4_linear(x, w, residual=x, drop=drop, seed=SEED, subsequence=subsequence(step, r, 1))
            error = y.float() - want.float()
            (error.square().sum() / (2 * tokens)).backward()
            loss += float(error.detach().square().mean()) / ranks
            grads.append(w.grad)
        if four_bits:
            sent = [rr.mx4_quantize(d, rounding="stochastic", seed=SEED, subsequence=subsequence(step, r, 3))
                    for r, d in enumerate(grads)]
            total = rr.mx4_allreduce(sent, dtype=torch.float32)
        else:
            total = rr.allreduce([d.float() for d in grads])
        for r in range(ranks):
            weights[r] = (weights[r].float() - 0.5 / ranks * total[r].view(features, features)).to(torch.bfloat16)
        losses.append(loss)
    # the ring gives every rank the same bits, so the replicas stay alike
    assert all(torch.equal(w, weights[0]) for w in weights)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--features", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    for four_bits, name in ((False, "binary32 wire"), (True, "4-bit wire")):
        losses = train(a.ranks, a.tokens, a.features, a.steps, four_bits)
        shown = ", ".join(f"{losses[i]:.4f}" for i in sorted({0, a.steps // 4, a.steps // 2, a.steps - 1}))
        print(f"{name}: loss {shown}")


if __name__ == "__main__":
    main()
