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
