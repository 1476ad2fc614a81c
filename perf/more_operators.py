"""Layer norm, the linear cross entropy and the orthogonalised update as measured cases.

Three kinds of case, each one pass of what a data-parallel training or serving
step does around its matrix products:

  norm   y = (x - mean) / sqrt(var + eps) * weight + bias over the rows of x,
         alone (serving) or with its backward pass: the gradients of x, weight
         and bias
  loss   the softmax cross entropy of logits = x W^T against one target a
         token, alone (scoring) or with the gradients of x and W; a token
         whose target is -100 counts nothing
  orth   an update (a matrix, or a batch of equal ones) brought near the
         orthogonal matrix that has its singular vectors, after the ranks'
         gradients are summed

Definitions.  norm: mean and variance (over the row, divided by its length);
with h = (x - mean) / sqrt(var + eps) and g = dy * weight,
dx = (g - mean(g) - h mean(g h)) / sqrt(var + eps), dweight = sum over rows of
dy h, dbias = sum over rows of dy.  loss: loss[t] = log(sum_v exp(l[t, v])) -
l[t, target[t]], and 0 for a token without a target; with p the softmax and
e[t, v] = grad * (p[t, v] - (v == target[t])), 0 for a token without one,
dx = e W and dW = e^T x; grad is the gradient that every token's loss has (one
over the tokens that count, and for binary16 times a loss scale).  orth:
X = G / (|G| + eps) in the Frobenius norm, then five times X <- a X + (b S +
c S^2) X with S = X X^T (X^T of the shorter side where G is tall) and (a, b, c)
= (3.4445, -4.7750, 2.0315).
"""
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NORM_EPS = 1e-5
ORTH_EPS = 1e-7
STEPS = 5
QUINTIC = (3.4445, -4.7750, 2.0315)
IGNORED = -100


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # one token's hidden state before a projection (serving, batch one)
        dict(name="norm_token", kind="norm", rows=1, cols=4096, dtype="bf16", weights="bf16", train=False),
        # a training micro-batch of hidden states, there and back
        dict(name="norm_train", kind="norm", rows=16384, cols=4096, dtype="bf16", weights="bf16", train=True),
        # odd sizes in binary32, there and back
        dict(name="norm_odd", kind="norm", rows=5003, cols=1999, dtype="f32", weights="f32", train=True),
        # the log-probability of one token over a large vocabulary (scoring while serving)
        dict(name="loss_token", kind="loss", tokens=1, hidden=4096, vocabulary=131072, dtype="bf16", train=False),
        # a few tokens of a small model, there and back
        dict(name="loss_short", kind="loss", tokens=33, hidden=1024, vocabulary=8000, dtype="bf16", train=True),
        # odd sizes in all three directions, with a loss scale
        dict(name="loss_odd", kind="loss", tokens=1003, hidden=777, vocabulary=5003, dtype="f16", train=True),
        # a training micro-batch over an ordinary vocabulary
        dict(name="loss_train", kind="loss", tokens=8192, hidden=4096, vocabulary=32000, dtype="bf16", train=True),
        # a smaller one over a large vocabulary
        dict(name="loss_vocabulary", kind="loss", tokens=2048, hidden=2048, vocabulary=131072, dtype="bf16", train=True),
        # the small projections of eight layers at once
        dict(name="orth_small", kind="orth", batch=8, rows=128, cols=512, dtype="f32"),
        # an odd-sized binary32 gradient
        dict(name="orth_odd", kind="orth", batch=1, rows=777, cols=1537, dtype="f32"),
        # a square projection's summed gradient
        dict(name="orth_square", kind="orth", batch=1, rows=4096, cols=4096, dtype="bf16"),
        # an up projection's, taller than wide
        dict(name="orth_tall", kind="orth", batch=1, rows=11008, cols=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _bounded(rng, most, *ranges):
    """Sizes of these ranges (over their logarithms) whose product is at most `most`."""
    sizes = [_log(rng, lo, hi) for lo, hi in ranges]
    total = 1
    for s in sizes:
        total *= s
    if total > most:
        big = max(range(len(sizes)), key=lambda j: sizes[j])
        sizes[big] = max(ranges[big][0], sizes[big] * most // total)
    return sizes


def draw(rng):
    kind = rng.choice(("norm", "norm", "loss", "loss", "orth"))
    if kind == "norm":
        rows, cols = _bounded(rng, 16384 * 4096, (1, 16384), (33, 16384))
        dtype = rng.choice(("f32", "f16", "bf16"))
        return dict(kind=kind, rows=rows, cols=cols, dtype=dtype, weights=rng.choice((dtype, "f32")), train=rng.random() < 0.75)
    if kind == "loss":
        tokens, hidden, vocabulary = _bounded(rng, 8192 * 4096 * 16000, (1, 8192), (64, 8192), (500, 131072))
        return dict(kind=kind, tokens=tokens, hidden=hidden, vocabulary=vocabulary, dtype=rng.choice(("f16", "bf16")),
                    train=rng.random() < 0.75)
    rows, cols = _bounded(rng, 4096 * 4096, (32, 8192), (32, 8192))
    return dict(kind=kind, batch=rng.choice((1, 1, 2, 3)), rows=rows, cols=cols, dtype=rng.choice(("f32", "f16", "bf16")))


def work(case):
    kind = case["kind"]
    if kind == "norm":
        n, s = case["rows"] * case["cols"], SIZE[case["dtype"]]
        w = 2 * case["cols"] * SIZE[case["weights"]]
        return {"bytes": 5 * n * s + 2 * w if case["train"] else 2 * n * s + w, "flops": (20 if case["train"] else 8) * n}
    if kind == "loss":
        t, h, v = case["tokens"], case["hidden"], case["vocabulary"]
        each = t * h + v * h
        return {"bytes": 2 * each * (3 if case["train"] else 1), "flops": 2 * t * h * v * (3 if case["train"] else 1)}
    m, n = sorted((case["rows"], case["cols"]))
    # S and its square are symmetric: half of each is enough
    return {"bytes": case["batch"] * m * n * (SIZE[case["dtype"]] + 2),
            "flops": case["batch"] * STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)}


# ----------------------------------------------------------------- the inputs


def _normal(g, shape, sigma):
    return torch.randn(shape, generator=g, device="cuda").mul_(sigma)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, s = case["kind"], dict(case)
    if kind == "norm":
        # hidden states with a mean of their own and a few columns far larger than the others
        t, shape = TYPES[case["dtype"]], (case["rows"], case["cols"])
        loud = (torch.rand((1, case["cols"]), generator=g, device="cuda") < 0.01).float()
        x = _normal(g, shape, 1.0).mul_(1 + 15 * loud)
        s["x"] = x.add_(_normal(g, (case["rows"], 1), 0.5)).to(t)
        del x
        s["weight"] = (1 + _normal(g, (case["cols"],), 0.1)).to(TYPES[case["weights"]])
        s["bias"] = _normal(g, (case["cols"],), 0.1).to(TYPES[case["weights"]])
        if case["train"]:
            s["dy"] = _normal(g, shape, 1e-2).to(t)
    elif kind == "loss":
        # hidden states that know something of their target, and targets that go by frequency;
        # a tenth of the tokens (of a prompt) count nothing
        t, n, h, v = TYPES[case["dtype"]], case["tokens"], case["hidden"], case["vocabulary"]
        w = _normal(g, (v, h), 0.02).to(t)
        target = (torch.rand((n,), generator=g, device="cuda") ** 3 * v).long().clamp_(max=v - 1)
        known = 4.0 * torch.rand((n, 1), generator=g, device="cuda") / (4e-4 * h)
        x = (_normal(g, (n, h), 1.0) + known * w[target].float()).to(t)
        target[torch.rand((n,), generator=g, device="cuda") < 0.1] = IGNORED
        target[0] = v // 3
        s["x"], s["w"], s["target"] = x, w, target
        kept = (target != IGNORED).sum().float()
        s["grad"] = 1 / kept if case["dtype"] == "bf16" else torch.full_like(kept, 4.0)  # (binary16: a loss scale of 4 * kept)
    else:
        # a gradient: a few strong directions and noise
        b, m, n = case["batch"], case["rows"], case["cols"]
        strong = _normal(g, (b, m, 16), 1.0) @ _normal(g, (b, 16, n), 0.25)
        s["g"] = strong.add_(_normal(g, (b, m, n), 0.3)).mul_(1e-2).to(TYPES[case["dtype"]])
        if b == 1:
            s["g"] = s["g"][0]
    return s


# ------------------------------------------------------------ the plain forms


def _plain(s):
    if s["kind"] == "norm":
        t, x = s["x"].dtype, s["x"].float()
        w, b = s["weight"].float(), s["bias"].float()
        c = x - x.mean(-1, keepdim=True)
        rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + NORM_EPS)
        h = c * rstd
        y = (h * w + b).to(t)
        if not s["train"]:
            return {"y": y}
        dy = s["dy"].float()
        g = dy * w
        dx = (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True)) * rstd
        wt = s["weight"].dtype
        return {"y": y, "dx": dx.to(t), "dweight": (dy * h).sum(0).to(wt), "dbias": dy.sum(0).to(wt)}
    if s["kind"] == "loss":
        t, x, w = s["x"].dtype, s["x"].float(), s["w"].float()
        l = x @ w.t()
        counts = s["target"] != IGNORED
        at = s["target"].clamp(min=0).unsqueeze(1)
        top = l.amax(1, keepdim=True)
        own_logit = l.gather(1, at)
        l = l.sub_(top).exp_()
        total = l.sum(1, keepdim=True)
        loss = torch.where(counts, (total.log() + top - own_logit).squeeze(1), 0.0)
        if not s["train"]:
            return {"loss": loss}
        e = l.div_(total).scatter_add_(1, at, torch.full_like(total, -1.0))
        e = e.mul_(torch.where(counts, s["grad"], 0.0).unsqueeze(1))
        return {"loss": loss, "dx": (e @ w).to(t), "dw": (e.t() @ x).to(t)}
    x = s["g"].float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-1, -2)
    x = x / ((x * x).sum((-1, -2), keepdim=True).sqrt() + ORTH_EPS)
    a, b, c = QUINTIC
    for _ in range(STEPS):
        q = x @ x.transpose(-1, -2)
        x = a * x + (b * q + c * (q @ q)) @ x
    return (x.transpose(-1, -2) if tall else x).to(torch.bfloat16)


# ------------------------------------------------------- the framework's calls


def _own(s):
    import ring_allreduce_reducescatter_gb300 as rr

    if s["kind"] == "norm":
        if not s["train"]:
            return {"y": rr.layer_norm(s["x"], s["weight"], s["bias"], eps=NORM_EPS)}
        y, mean, rstd = rr.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=NORM_EPS)
        dx, dweight, dbias = rr.layer_norm_backward(s["dy"], s["x"], mean, rstd, s["weight"])
        return {"y": y, "dx": dx, "dweight": dweight, "dbias": dbias}
    if s["kind"] == "loss":
        if not s["train"]:
            return {"loss": rr.linear_cross_entropy(s["x"], s["w"], s["target"], ignore_index=IGNORED, reduction="none")}
        loss, lse = rr.linear_cross_entropy_forward(s["x"], s["w"], s["target"], ignore_index=IGNORED)
        dx, dw = rr.linear_cross_entropy_backward(s["grad"], s["x"], s["w"], s["target"], lse, ignore_index=IGNORED)
        return {"loss": loss, "dx": dx, "dw": dw}
    return rr.orthogonalize(s["g"], steps=STEPS, eps=ORTH_EPS, dtype=torch.bfloat16)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        n = x.shape[1]
        mean = torch.einsum("rc->r", x) / n
        var = torch.einsum("rc,rc->r", x, x) / n - mean ** 2
        inv = 1.0 / torch.sqrt(var + NORM_EPS)
        h = torch.einsum("rc,r->rc", x - mean[:, None], inv)
        y = torch.addcmul(b, h, w)
        if not case["train"]:
            return {"y": y}
        dy = s["dy"].double()
        s1, s2 = torch.einsum("rc,c->r", dy, w) / n, torch.einsum("rc,c,rc->r", dy, w, h) / n
        dx = (dy * w - s1[:, None] - s2[:, None] * h) * inv[:, None]
        return {"y": y, "dx": dx, "dweight": torch.einsum("rc,rc->c", dy, h), "dbias": torch.einsum("rc->c", dy)}
    if case["kind"] == "loss":
        x, w, target = s["x"].double(), s["w"].double(), s["target"]
        n, v = x.shape[0], w.shape[0]
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        loss = torch.zeros(n, dtype=torch.float64, device=x.device)
        part = max(1, (1 << 28) // v)
        for r in range(0, n, part):
            l = torch.einsum("th,vh->tv", x[r:r + part], w)
            lse = torch.logsumexp(l, 1)
            here = target[r:r + part]
            rows = (here != IGNORED).nonzero().squeeze(1)
            at = here[rows]
            loss[r + rows] = lse[rows] - l[rows, at]
            if case["train"]:
                e = torch.zeros_like(l)
                e[rows] = torch.exp(l[rows] - lse[rows, None])
                e[rows, at] -= 1
                e *= s["grad"].double()
                dx[r:r + part] = torch.einsum("tv,vh->th", e, w)
                dw += torch.einsum("tv,th->vh", e, x[r:r + part])
        return {"loss": loss, "dx": dx, "dw": dw} if case["train"] else {"loss": loss}
    # the singular vectors stay, the values go through the polynomial: X p(X^T X) on the shorter side
    g = s["g"].double()
    tall = g.shape[-2] >= g.shape[-1]
    x = g / (torch.linalg.matrix_norm(g).unsqueeze(-1).unsqueeze(-1) + ORTH_EPS)
    i = torch.eye(min(g.shape[-2:]), dtype=torch.float64, device=g.device)
    a, b, c = QUINTIC
    gram = torch.matmul(x.mT, x) if tall else torch.matmul(x, x.mT)
    whole = i.expand_as(gram)
    for _ in range(STEPS):  # (every factor is a polynomial of the first Gram matrix: they commute)
        p = a * i + torch.matmul(gram, b * i + c * gram)
        whole = torch.matmul(whole, p)
        gram = torch.matmul(torch.matmul(p, gram), p)
    return torch.matmul(x, whole) if tall else torch.matmul(whole, x)
