"""Data-parallel training of a small next-token model over R virtual ranks.

Every rank embeds its tokens, normalises them, runs the 4-bit layer h = x +
dropout(norm(x) W^T), normalises again and takes the softmax cross entropy of the
next token, whose logits are never stored.  The ranks' gradients are summed by the
ring AllReduce; the layer's matrix takes an orthogonalised step of its momentum
(as the Muon optimiser does), the output matrix and the norms plain ones.

    python examples/muon_data_parallel.py [--ranks 4] [--tokens 512] [--features 256] [--vocabulary 1000] [--steps 40]

Prints the mean loss as it goes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_allreduce_reducescatter_gb300 as rr  # noqa: E402

SEED = 2025
BF16 = torch.bfloat16


def parameters(features: int, vocabulary: int, seed: int = 1):
    """The embedding (not trained), the layer's matrix, the output matrix and the norms' weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    return {"embedding": r(vocabulary, features).to(BF16), "layer": (r(features, features) / features ** 0.5).to(BF16),
            "output": (r(vocabulary, features) / features ** 0.5).to(BF16), "norm1": torch.ones(features, device="cuda"),
            "bias1": torch.zeros(features, device="cuda"), "norm2": torch.ones(features, device="cuda")}


TRAINED = ("layer", "output", "norm1", "bias1", "norm2")


def loss_of(p, tokens, target, drop=None, seed=0, subsequence=0):
    """The mean loss of one rank's micro-batch."""
    x = p["embedding"][tokens]
    h = rr.mx4_linear(rr.layer_norm(x, p["norm1"], p["bias1"]), p["layer"], residual=x, drop=drop, seed=seed,
                      subsequence=subsequence)
    return rr.linear_cross_entropy(rr.layer_norm(h, p["norm2"]), p["output"], target)


def gradients(p, tokens, target, **how):
    """(loss, the trained parameters' gradients)."""
    q = {k: (v.detach().requires_grad_() if k in TRAINED else v) for k, v in p.items()}
    loss = loss_of(q, tokens, target, **how)
    return loss.detach(), dict(zip(TRAINED, torch.autograd.grad(loss, [q[k] for k in TRAINED])))


def train(ranks: int, tokens: int, features: int, vocabulary: int, steps: int, p_drop: float = 0.1):
    p = parameters(features, vocabulary)
    g = torch.Generator(device="cuda").manual_seed(2)
    follows = torch.randperm(vocabulary, generator=g, device="cuda")  # the token after each token
    momentum = torch.zeros((features, features), device="cuda")
    losses = []
    for step in range(steps):
        mean, each = 0.0, []
        for r in range(ranks):
            here = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
            there = follows[here]
            there[: tokens // 16] = -100  # (a prompt counts nothing)
            sub = (step * 64 + r) * 4
            loss, grads = gradients(p, here, there, drop=rr.Dropout(p_drop, SEED, sub), seed=SEED, subsequence=sub + 1)
            mean += float(loss) / ranks
            each.append(grads)
        total = {k: rr.allreduce([e[k].float().reshape(-1) for e in each])[0].view(p[k].shape) / ranks for k in TRAINED}
        momentum.mul_(0.9).add_(total["layer"])
        p["layer"] = (p["layer"].float() - 0.02 * rr.orthogonalize(momentum)).to(BF16)
        p["output"] = (p["output"].float() - 2.0 * total["output"]).to(BF16)
        for k in ("norm1", "bias1", "norm2"):
            p[k] = p[k] - 0.1 * total[k]
        losses.append(mean)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--features", type=int, default=256)
    ap.add_argument("--vocabulary", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args()
    losses = train(a.ranks, a.tokens, a.features, a.vocabulary, a.steps)
    print("loss " + ", ".join(f"{losses[i]:.4f}" for i in sorted({0, a.steps // 4, a.steps // 2, a.steps - 1})))


if __name__ == "__main__":
    main()
