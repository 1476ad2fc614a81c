"""Layer norm, the linear cross entropy and the orthogonalised update in 64 bits,
for the tests: written from the definitions in include/ringred.h, sharing nothing
with the kernels."""
import torch

U = 2.0 ** -24  # half a step of binary32, relative


def half_step(dtype) -> float:
    """The largest relative error of one rounding to this format."""
    return torch.finfo(dtype).eps / 2


def norm(x, weight, bias, eps):
    """(y, mean, rstd, h)."""
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    h = (x - mean) * rstd
    y = h if weight is None else h * weight.double()
    return y if bias is None else y + bias.double(), mean.squeeze(-1), rstd.squeeze(-1), h


def norm_grad(dy, x, mean, rstd, weight):
    """(dx, dweight, dbias) with the mean and rstd given."""
    dy, h = dy.double(), (x.double() - mean.double().unsqueeze(-1)) * rstd.double().unsqueeze(-1)
    g = dy if weight is None else dy * weight.double()
    dx = (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True)) * rstd.double().unsqueeze(-1)
    axes = tuple(range(dy.dim() - 1))
    return dx, (dy * h).sum(axes), dy.sum(axes)


def cross_entropy(x, w, target, ignore_index):
    """(loss, lse, logits)."""
    l = x.double() @ w.double().t()
    lse = torch.logsumexp(l, 1)
    counts = target != ignore_index
    at = torch.where(counts, target, 0)
    return torch.where(counts, lse - l.gather(1, at[:, None]).squeeze(1), 0.0), lse, l


def cross_entropy_grad(grad, l, target, ignore_index):
    """e: the gradient of the logits; grad: one element, or one a token."""
    counts = target != ignore_index
    e = torch.softmax(l, 1)
    e[torch.arange(l.shape[0], device=l.device), torch.where(counts, target, 0)] -= 1
    return e * (torch.where(counts, 1.0, 0.0) * grad.double())[:, None]


QUINTIC = (3.4445, -4.7750, 2.0315)
HELD = (2.0 ** 6, 2.0 ** 14, 2.0 ** 13)  # what X, S and b S + c S^2 are held times


def orthogonal(g, steps, eps, held=False):
    """Newton-Schulz steps in 64 bits; held: with X, S and the polynomial rounded to binary16 as the kernels hold them."""
    def keep(t, scale):
        return (t * scale).half().double() / scale if held else t

    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = keep(x / (torch.linalg.matrix_norm(x).unsqueeze(-1).unsqueeze(-1) + eps), HELD[0])
    a, b, c = QUINTIC
    for k in range(steps):
        s = keep(x @ x.mT, HELD[1])
        p = keep(b * s + c * (s @ s), HELD[2])
        x = a * x + p @ x
        if k + 1 < steps:
            x = keep(x, HELD[0])
    return x.mT if tall else x
