"""The linear cross entropy and its gradient against the definition in 64 bits.

Tolerances.  u = 2^-24.  A product over K on the tensor cores takes ceil(K / 16)
steps, each of which may cut its sum to binary32: an element is off by at most
2^-22 (ceil(K / 16) + 4) times its sum of magnitudes.  With d the largest such
error of a row's logits: the exponentials (2 u, and their argument's rounding u
|l - m|), their sums (a tree of at most 64 + vocabulary / 64 additions) and the
logarithm leave lse off by d + D u + 2 u |lse|, a loss by twice that and d.  In e
a probability is off, relative, by twice d, D u, u |l - lse|, and half a step of
the storage format; dx and dw are products of e, rounded once."""
import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = ref.U


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import ring_allreduce_reducescatter_gb300 as mod

    torch.cuda.set_device(0)
    return mod


def draw(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def inputs(tokens, hidden, vocabulary, dtype, seed=1, ignored=0.2, logits=2.0):
    x = draw((tokens, hidden), seed, dtype)
    w = draw((vocabulary, hidden), seed + 1, dtype, logits / hidden ** 0.5)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    target = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
    target[torch.rand(tokens, generator=g, device="cuda") < ignored] = -100
    return x, w, target


def product_error(k):
    return 2.0 ** -22 * (-(-k // 16) + 4)


def lse_error(x, w, lse):
    """(the largest error of a row's logits, of its lse)."""
    d = product_error(x.shape[1]) * (x.double().abs() @ w.double().abs().t()).amax(1)
    spread = 64 + w.shape[0] // 64 + 4
    return d, 1.01 * (d + (spread + 60) * U + 2 * U * lse.abs())


def check_losses(loss, lse, x, w, target, ignore=-100):
    want, want_lse, l = ref.cross_entropy(x, w, target, ignore)
    d, off = lse_error(x, w, want_lse)
    if lse is not None:
        assert ((lse.double() - want_lse).abs() <= off).all()
    assert ((loss.double() - want).abs() <= 2 * off + d + U * want.abs()).all()
    assert (loss[target == ignore] == 0).all()
    return l


def check_gradients(dx, dw, grad, x, w, target, l, ignore=-100):
    dtype, xd, wd = x.dtype, x.double(), w.double()
    e = ref.cross_entropy_grad(grad, l, target, ignore)
    d, off = lse_error(x, w, torch.logsumexp(l, 1))
    p = torch.softmax(l, 1)
    g = (torch.where(target != ignore, 1.0, 0.0) * grad.double().abs())[:, None]
    # of p: the logit, lse and the exponential; then e's rounding
    off_e = g * p * ((2 * d + off)[:, None] + 64 * U) + 4 * U * e.abs()
    off_e = off_e + ref.half_step(dtype) * (e.abs() + off_e) + g.max() * 2.0 ** -38  # (a subnormal of binary16, scaled)
    top = torch.finfo(dtype)
    for out, want, size, spread, k in ((dx, e @ wd, e.abs() @ wd.abs(), off_e @ wd.abs(), w.shape[0]),
                                       (dw, e.t() @ xd, e.abs().t() @ xd.abs(), off_e.t() @ xd.abs(), x.shape[0])):
        if out is None:
            continue
        bound = 1.01 * (spread + product_error(k) * (size + spread))
        bound = bound + top.eps / 2 * (want.abs() + bound) + top.tiny * top.eps
        # (a value that rounds past the format's largest is infinity)
        past = (want.abs() + bound > top.max) & (out == torch.copysign(torch.full_like(want, float("inf")), want))
        assert ((out.double() - want).abs() <= bound)[~past].all()
        # and well inside it on the whole: roundings of many terms do not add up
        if want.numel() > 1000 and not past.any():
            assert (out.double() - want).norm() <= 2 * ref.half_step(dtype) * want.norm()


SHAPES = [(1, 64, 500), (1, 1, 1), (3, 8, 2), (5, 16, 64), (33, 129, 1000), (128, 64, 130), (129, 64, 257), (130, 777, 523),
          (300, 96, 5003), (1000, 200, 129), (257, 72, 20000), (64, 1024, 8000), (2500, 320, 2500), (2300, 2320, 2330)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,hidden,vocabulary", SHAPES)
def test_losses(rr, tokens, hidden, vocabulary, dtype):
    x, w, target = inputs(tokens, hidden, vocabulary, dtype)
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    torch.cuda.synchronize()
    assert rr.device_status() == 0
    check_losses(loss, lse, x, w, target)
    assert torch.equal(rr.linear_cross_entropy(x, w, target, reduction="none"), loss)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,hidden,vocabulary", SHAPES)
def test_gradients(rr, tokens, hidden, vocabulary, dtype):
    x, w, target = inputs(tokens, hidden, vocabulary, dtype)
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    l = check_losses(loss, lse, x, w, target)
    each = draw(tokens, 7).abs() + 0.1
    for grad in (torch.full((), 0.5, device="cuda"), each):
        dx, dw = rr.linear_cross_entropy_backward(grad, x, w, target, lse)
        torch.cuda.synchronize()
        assert rr.device_status() == 0
        check_gradients(dx, dw, grad, x, w, target, l)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_pieces_of_the_vocabulary(rr, dtype):
    """More than 2^27 elements of logits: two pieces, the last of an odd width."""
    x, w, target = inputs(8200, 72, 17001, dtype)
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    l = check_losses(loss, lse, x, w, target)
    grad = torch.full((), 1.0 / 64, device="cuda")
    dx, dw = rr.linear_cross_entropy_backward(grad, x, w, target, lse)
    check_gradients(dx, dw, grad, x, w, target, l)


@pytest.mark.parametrize("scale", [2.0 ** -30, 1e-6, 3.0, 2.0 ** 14])
def test_small_and_large_gradients_in_binary16(rr, scale):
    """The common power of two keeps e inside binary16; outputs are checked where binary16 holds them."""
    x, w, target = inputs(100, 96, 700, F16)
    w = w * 64 if scale < 1 else w / 64
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    l = ref.cross_entropy(x, w, target, -100)[2]
    grad = torch.full((), scale, device="cuda")
    dx, dw = rr.linear_cross_entropy_backward(grad, x, w, target, lse)
    check_gradients(dx, dw, grad, x, w, target, l) if scale >= 1 else None
    e = ref.cross_entropy_grad(grad, l, target, -100)
    want = e.t() @ x.double()
    held = want.abs() < 65000  # binary16's largest is 65504
    assert dx.isfinite().all() and dw[held].isfinite().all()
    assert ((dw.double() - want).abs() <= 2.0 ** -24 + 0.02 * (e.abs().t() @ x.double().abs()))[held].all()


@pytest.mark.parametrize("x_pad,w_pad,at", [(8, 16, 0), (1, 0, 0), (0, 3, 0), (8, 8, 4), (5, 7, 1)])
@pytest.mark.parametrize("tokens,hidden", [(150, 96), (600, 1024)])
def test_strides(rr, tokens, hidden, x_pad, w_pad, at):
    """Rows of wider arrays: read as they lie on the 16-byte grid, through a copy off it."""
    x, w, target = inputs(tokens, hidden, 700, BF16)
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    grad = torch.full((), 0.5, device="cuda")
    want = (loss, lse) + rr.linear_cross_entropy_backward(grad, x, w, target, lse)

    def held(t, pad):
        whole = torch.full((t.shape[0], t.shape[1] + pad + at), float("nan"), dtype=t.dtype, device="cuda")
        whole[:, at:at + t.shape[1]] = t
        return whole[:, at:at + t.shape[1]]

    xs, ws = held(x, x_pad), held(w, w_pad)
    loss, lse = rr.linear_cross_entropy_forward(xs, ws, target)
    got = (loss, lse) + rr.linear_cross_entropy_backward(grad, xs, ws, target, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tokens", [70, 300])
def test_outputs_in_wider_rows_leave_the_rest(rr, tokens):
    import ctypes

    hidden, vocabulary = 100, 333
    x, w, target = inputs(tokens, hidden, vocabulary, BF16)
    _, lse = rr.linear_cross_entropy_forward(x, w, target)
    grad = torch.full((), 0.5, device="cuda")
    want = rr.linear_cross_entropy_backward(grad, x, w, target, lse)
    L = rr.lib()
    for pad in (28, 5):
        dx = torch.full((tokens + 3, hidden + pad), 7.0, dtype=BF16, device="cuda")
        dw = torch.full((vocabulary + 3, hidden + pad), 7.0, dtype=BF16, device="cuda")
        need = L.ring_linear_cross_entropy_backward_workspace(x.data_ptr(), hidden, w.data_ptr(), hidden, tokens, hidden, vocabulary)
        space = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
        st = L.ring_linear_cross_entropy_backward(grad.data_ptr(), 0, x.data_ptr(), hidden, w.data_ptr(), hidden, target.data_ptr(),
                                                  -100, lse.data_ptr(), dx.data_ptr(), hidden + pad, dw.data_ptr(), hidden + pad,
                                                  tokens, hidden, vocabulary, 2, space.data_ptr(), need,
                                                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        assert (space[need:] == 7).all()
        for got, ref_, rows in ((dx, want[0], tokens), (dw, want[1], vocabulary)):
            assert torch.equal(got[:rows, :hidden], ref_)
            assert (got[rows:] == 7).all() and (got[:, hidden:] == 7).all()


def test_tokens_that_do_not_count(rr):
    """All of them, all but one, and an ignored index inside the vocabulary; logits of an ignored token may be no numbers."""
    x, w, target = inputs(200, 64, 300, BF16, ignored=0.0)
    none = torch.full_like(target, -100)
    for reduction, empty in (("mean", 0.0), ("sum", 0.0)):
        assert rr.linear_cross_entropy(x, w, none, reduction=reduction).item() == empty
    loss, lse = rr.linear_cross_entropy_forward(x, w, none)
    assert (loss == 0).all()
    dx, dw = rr.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, none, lse)
    assert (dx == 0).all() and (dw == 0).all()
    one = none.clone()
    one[77] = 5
    loss, lse = rr.linear_cross_entropy_forward(x, w, one)
    l = check_losses(loss, lse, x, w, one)
    assert rr.linear_cross_entropy(x, w, one) == loss[77]
    grad = torch.ones((), device="cuda")
    dx, dw = rr.linear_cross_entropy_backward(grad, x, w, one, lse)
    check_gradients(dx, dw, grad, x, w, one, l)
    loss = rr.linear_cross_entropy(x, w, target, ignore_index=7, reduction="none")
    check_losses(loss, None, x, w, target, 7)
    x2 = x.clone()
    x2[3] = float("nan")
    t2 = target.clone()
    t2[3] = -100
    loss, lse = rr.linear_cross_entropy_forward(x2, w, t2)
    assert loss[3] == 0 and loss.isfinite().all()
    dx, _ = rr.linear_cross_entropy_backward(grad, x2, w, t2, lse, want_dw=False)
    assert (dx[3] == 0).all() and dx.isfinite().all()


def test_targets_outside_the_vocabulary(rr):
    x, w, target = inputs(200, 64, 300, BF16, ignored=0.0)
    clean = rr.linear_cross_entropy(x, w, target, reduction="none")
    target[3], target[9], target[150] = 300, -1, 1 << 40
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    bad = torch.zeros(200, dtype=torch.bool, device="cuda")
    bad[[3, 9, 150]] = True
    assert loss[bad].isnan().all() and torch.equal(loss[~bad], clean[~bad])
    dx, dw = rr.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, target, lse)
    assert dx[bad].isnan().all() and dx[~bad].isfinite().all() and dw.isnan().all()


def test_not_finite_logits(rr):
    x, w, target = inputs(200, 64, 300, BF16, ignored=0.0)
    clean = rr.linear_cross_entropy(x, w, target, reduction="none")
    x[5], x[140, 3] = float("inf"), float("nan")
    loss = rr.linear_cross_entropy(x, w, target, reduction="none")
    rest = [i for i in range(200) if i not in (5, 140)]
    assert loss[[5, 140]].isnan().all() and torch.equal(loss[rest], clean[rest])


def test_large_logits(rr):
    """Probabilities of one and zero: the maximum comes off before the exponential."""
    x, w, target = inputs(140, 64, 300, BF16, logits=300.0)
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    check_losses(loss, lse, x, w, target)
    dx, dw = rr.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, target, lse)
    assert dx.isfinite().all() and dw.isfinite().all()


def test_parts_and_no_tokens(rr):
    x, w, target = inputs(150, 64, 300, BF16)
    _, lse = rr.linear_cross_entropy_forward(x, w, target)
    grad = torch.full((), 0.5, device="cuda")
    dx, dw = rr.linear_cross_entropy_backward(grad, x, w, target, lse)
    a, none = rr.linear_cross_entropy_backward(grad, x, w, target, lse, want_dw=False)
    assert torch.equal(a, dx) and none is None
    none, b = rr.linear_cross_entropy_backward(grad, x, w, target, lse, want_dx=False)
    assert torch.equal(b, dw) and none is None
    x, target = x[:0], target[:0]
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    assert loss.shape == (0,) and rr.linear_cross_entropy(x, w, target).item() == 0
    dx, dw = rr.linear_cross_entropy_backward(grad, x, w, target, lse)
    assert dx.shape == (0, 64) and (dw == 0).all() and dw.shape == w.shape


def test_past_four_billion_elements(rr):
    """Rows of w and dw beyond element 2^32: all rows but the first and last thousand are zero, their logits 0."""
    tokens, hidden, vocabulary, k = 130, 4096, (1 << 20) + 5000, 1000
    w = torch.zeros((vocabulary, hidden), dtype=BF16, device="cuda")
    w[:k], w[-k:] = draw((k, hidden), 1, BF16, 0.05), draw((k, hidden), 2, BF16, 0.05)
    x = draw((tokens, hidden), 3, BF16)
    target = torch.randint(0, vocabulary, (tokens,), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    target[::2] = vocabulary - 1 - torch.arange(65, device="cuda") * 7
    ends = torch.cat((w[:k], w[-k:]))
    l = x.double() @ ends.double().t()
    lse = (l.exp().sum(1) + (vocabulary - 2 * k)).log()
    at = torch.where(target < k, target, target - vocabulary + 2 * k)  # in `ends`, where it is there
    there = (target < k) | (target >= vocabulary - k)
    chosen = torch.where(there, l.gather(1, at.clamp(0, 2 * k - 1)[:, None]).squeeze(1), 0.0)
    loss, got = rr.linear_cross_entropy_forward(x, w, target)
    d, off = lse_error(x, ends, lse)
    off = off + (vocabulary // 64) * U
    assert ((got.double() - lse).abs() <= off).all()
    assert ((loss.double() - (lse - chosen)).abs() <= 2 * off + d).all()
    dx, dw = rr.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, target, got)
    e = torch.exp(l - lse[:, None])
    rows = torch.arange(tokens, device="cuda")[there]
    e[rows, at[there]] -= 1
    want = e.t() @ x.double()
    for part, here in ((dw[:k], want[:k]), (dw[-k:], want[-k:])):
        assert (part.double() - here).norm() <= 2 * ref.half_step(BF16) * here.norm()
    assert (dx.double() - e @ ends.double()).norm() <= 2 * ref.half_step(BF16) * (e @ ends.double()).norm()
    middle = int(target[~there][0])
    one = (e.new_zeros(hidden) + (torch.exp(-lse)[:, None] * x.double()).sum(0)) - x[target == middle].double().sum(0)
    assert (dw[middle].double() - one).norm() <= 2 * ref.half_step(BF16) * one.norm()
    del w, dw
    torch.cuda.empty_cache()


def test_same_bits_every_time(rr):
    x, w, target = inputs(1000, 200, 3000, BF16)
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    grad = torch.full((), 0.5, device="cuda")
    first = (loss, lse) + rr.linear_cross_entropy_backward(grad, x, w, target, lse)
    for _ in range(5):
        loss, lse = rr.linear_cross_entropy_forward(x, w, target)
        assert all(torch.equal(a, b) for a, b in zip((loss, lse) + rr.linear_cross_entropy_backward(grad, x, w, target, lse), first))


# ------------------------------------------------------------------- autograd


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_autograd(rr, reduction):
    x, w, target = inputs(150, 64, 300, BF16)
    x.requires_grad_(), w.requires_grad_()
    out = rr.linear_cross_entropy(x, w, target, reduction=reduction)
    up = draw(150, 9) if reduction == "none" else torch.tensor(2.0, device="cuda")
    out.backward(up)
    with torch.no_grad():
        loss, lse = rr.linear_cross_entropy_forward(x, w, target)
        count = (target != -100).sum().float()
        grad = up / count if reduction == "mean" else up
        want = rr.linear_cross_entropy_backward(grad, x, w, target, lse)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])
    value = loss if reduction == "none" else loss.double().sum() if reduction == "sum" else loss.double().sum() / count
    assert torch.allclose(out.detach().double(), value.double(), rtol=150 * U, atol=0)


def test_gradient_against_differences(rr):
    """Central differences of the kernel's loss, the steps exact in binary16: off by the product's error over h, by h^2 / 6
    times the third derivative (at most the largest change of a logit, cubed), and by e's rounding."""
    x, w, target = inputs(60, 64, 200, F16, logits=1.0)
    loss, lse = rr.linear_cross_entropy_forward(x, w, target)
    dx, dw = rr.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, target, lse)
    h = 2.0 ** -4
    for t, g, seed in ((x, dx, 5), (w, dw, 6)):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        v = torch.zeros_like(t)
        at = torch.randint(0, t.shape[1], (t.shape[0],), generator=gen, device="cuda")
        v[torch.arange(t.shape[0], device="cuda"), at] = h
        up, down = t + v, t - v
        step = (up.double() - down.double()) / 2  # what the steps came to in binary16
        a, b = ((up, w), (down, w)) if t is x else ((x, up), (x, down))
        got = [rr.linear_cross_entropy(*args, target, reduction="none").double().sum().item() for args in (a, b)]
        slope = (got[0] - got[1]) / 2
        want = (g.double() * step).sum().item()
        change = (step.abs() @ w.double().abs().t() if t is x else x.double().abs() @ step.abs().t()).amax(1)
        noise = sum(3 * lse_error(*args, lse)[1].sum().item() for args in (a, b)) / 2
        skew = (change ** 3).sum().item() / 6
        rounding = 2.0 ** -10 * (g.double().abs() * step.abs()).sum().item() + 2.0 ** -11 * change.sum().item() * 2
        assert abs(slope - want) <= noise + skew + rounding


def test_refusals(rr):
    x, w, target = inputs(20, 64, 300, BF16)
    _, lse = rr.linear_cross_entropy_forward(x, w, target)
    one = torch.ones((), device="cuda")
    f, b = rr.linear_cross_entropy, rr.linear_cross_entropy_backward
    for call in (lambda: f(x.float(), w.float(), target), lambda: f(x, w.half(), target), lambda: f(x[:, :32], w, target),
                 lambda: f(x, w, target.int()), lambda: f(x, w, target[:19]), lambda: f(x.cpu(), w, target),
                 lambda: f(x, w, target.cpu()), lambda: f(x, w, target, reduction="max"), lambda: f(x.t(), w, target),
                 lambda: f(x[:, :0], w[:, :0], target), lambda: f(x, w[:0], target),
                 lambda: rr.linear_cross_entropy_forward(x.clone().requires_grad_(), w, target),
                 lambda: b(one.double(), x, w, target, lse), lambda: b(torch.ones(3, device="cuda"), x, w, target, lse),
                 lambda: b(one, x, w, target, lse[:5]), lambda: b(one, x, w, target, lse.half())):
        with pytest.raises(ValueError):
            call()


def test_another_stream_and_graphs(rr):
    """A graph replayed over new inputs, and two graphs of the same call in turn, each with its own workspace."""
    x, w, target = inputs(300, 64, 700, BF16)
    grad = torch.full((), 0.5, device="cuda")

    def step(x, w, target, **how):
        loss, lse = rr.linear_cross_entropy_forward(x, w, target, **how)
        return (loss, lse) + rr.linear_cross_entropy_backward(grad, x, w, target, lse, **how)

    want = step(x, w, target)
    x2, w2, target2 = inputs(300, 64, 700, BF16, seed=11)
    want2 = step(x2, w2, target2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(x, w, target, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    xs, ws, ts = x.clone(), w.clone(), target.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(xs, ws, ts)
        graphs.append((g, out))
    for a, b, c, expect in ((x2, w2, target2, want2), (x, w, target, want)):
        xs.copy_(a), ws.copy_(b), ts.copy_(c)
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, out in graphs:
            assert all(torch.equal(p, q) for p, q in zip(out, expect))
