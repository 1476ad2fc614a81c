"""What the differentiable 4-bit layer and dropout keep for their backward pass,
and which calls record a gradient."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import ring_allreduce_reducescatter_gb300 as mod

    torch.cuda.set_device(0)
    return mod


def draw(rows, cols, seed, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, cols), generator=g).to(dtype).cuda()


# ------------------------------------------------------------------- the layer


@pytest.mark.parametrize("need_x,need_w", [(True, True), (True, False), (False, True)])
def test_a_second_backward_pass_is_refused(rr, need_x, need_w):
    """Unless the graph was asked to stay; then it adds the same gradients again."""
    x, w, dy = draw(70, 96, 1), draw(130, 96, 2), draw(70, 130, 3)
    x.requires_grad_(need_x), w.requires_grad_(need_w)
    y = rr.mx4_linear(x, w, seed=4, subsequence=10)
    y.backward(dy, retain_graph=True)
    once = [t.grad.clone() for t in (x, w) if t.grad is not None]
    y.backward(dy)
    for t, g in zip([t for t in (x, w) if t.grad is not None], once):
        assert torch.equal(t.grad, 2 * g)
    with pytest.raises(RuntimeError, match="second time"):
        y.backward(dy)


def test_nothing_is_kept_after_the_backward_pass(rr):
    """With the output still held, only it and the gradients are left."""
    x, w = draw(1024, 2048, 1).requires_grad_(), draw(512, 2048, 2).requires_grad_()
    dy = draw(1024, 512, 3)
    x.grad, w.grad = torch.zeros_like(x), torch.zeros_like(w)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = rr.mx4_linear(x, w)
    own = y.numel() * y.element_size()
    assert torch.cuda.memory_allocated() - before > own  # the transposes, for the backward pass
    y.backward(dy)
    assert torch.cuda.memory_allocated() - before == own


def test_saved_tensor_hooks_see_what_is_kept(rr):
    x, w, dy = draw(70, 96, 1).requires_grad_(), draw(130, 96, 2).requires_grad_(), draw(70, 130, 3)
    rr.mx4_linear(x, w, seed=4, subsequence=10).backward(dy)
    want, x.grad, w.grad = (x.grad, w.grad), None, None
    seen = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: seen.append(t.numel()) or t, lambda t: t):
        y = rr.mx4_linear(x, w, seed=4, subsequence=10)
    # 96 rows of 3 blocks and 1 x 1 scale tiles; 96 rows of 5 blocks and 1 x 1
    assert sorted(seen) == [96 * 48 + 1024, 96 * 80 + 1024]
    y.backward(dy)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])


@pytest.mark.parametrize("how", ["host", "recompute"])
def test_kept_tensors_offloaded_or_computed_again(rr, how):
    x, w, dy = draw(300, 160, 1).requires_grad_(), draw(200, 160, 2).requires_grad_(), draw(300, 200, 3)
    layer = lambda a, b: rr.mx4_linear(a, b, drop=rr.Dropout(0.2, 9, 1), seed=4, subsequence=10)
    layer(x, w).backward(dy)
    want, x.grad, w.grad = (x.grad, w.grad), None, None
    if how == "host":
        with torch.autograd.graph.save_on_cpu():
            y = layer(x, w)
    else:
        from torch.utils.checkpoint import checkpoint

        y = checkpoint(layer, x, w, use_reentrant=False)
    y.backward(dy)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])


def test_a_layer_of_which_only_the_residual_learns(rr):
    """Nothing is kept for it, so its backward pass may be repeated, like an addition's."""
    x, w, r, dy = draw(40, 64, 1), draw(50, 64, 2), draw(40, 50, 3).requires_grad_(), draw(40, 50, 4)
    y = rr.mx4_linear(x, w, residual=r)
    y.backward(dy, retain_graph=True)
    y.backward(dy)
    assert torch.equal(r.grad, 2 * dy)


# --------------------------------------------------------------------- dropout


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shape", [(1,), (1000,), (33, 45), (3, 5, 7), (64, 256)])
def test_dropout_records_its_gradient(rr, shape, dtype):
    """dx is dropout(dy) with the same mask, the residual's gradient dy itself; the values are those without."""
    g = torch.Generator().manual_seed(1)
    x, r, dy = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(3))
    d = rr.Dropout(0.3, 8, 2, 5)
    plain, with_r = rr.dropout(x, d), rr.dropout(x, d, residual=r)
    x.requires_grad_(), r.requires_grad_()
    y = rr.dropout(x, d)
    assert y.requires_grad and torch.equal(y.detach(), plain)
    y.backward(dy)
    assert torch.equal(x.grad, rr.dropout(dy, d))
    x.grad = None
    y = rr.dropout(x, d, residual=r)
    assert torch.equal(y.detach(), with_r)
    y.backward(dy)
    assert torch.equal(x.grad, rr.dropout(dy, d)) and torch.equal(r.grad, dy)
    x.grad = r.grad = None
    rr.dropout(x.detach(), d, residual=r).backward(dy)
    assert x.grad is None and torch.equal(r.grad, dy)


def test_dropout_gradients_of_any_layout(rr):
    """A strided input, and gradients that are one value spread out or come transposed."""
    d = rr.Dropout(0.25, 5)
    whole = draw(33, 60, 1, F32).requires_grad_()
    y = rr.dropout(whole[:, 3:48], d)
    y.sum().backward()
    want = torch.zeros_like(whole)
    want[:, 3:48] = rr.dropout(torch.ones((33, 45), device="cuda"), d)
    assert torch.equal(whole.grad, want)
    x, dy = draw(33, 45, 2, F32).requires_grad_(), draw(45, 33, 3, F32)
    rr.dropout(x, d).backward(dy.t())
    assert torch.equal(x.grad, rr.dropout(dy.t().contiguous(), d))


def test_dropout_gradient_of_the_gradient(rr):
    """dropout is linear in x: the gradient with respect to dy of <dx, v> is dropout(v)."""
    d, x, v = rr.Dropout(0.25, 5), draw(9, 40, 1, F32).requires_grad_(), draw(9, 40, 2, F32)
    dy = draw(9, 40, 3, F32).requires_grad_()
    dx, = torch.autograd.grad(rr.dropout(x, d), x, dy, create_graph=True)
    dx.backward(v)
    assert torch.equal(dy.grad, rr.dropout(v, d))


def test_dropout_inside_a_model(rr):
    """A gradient passes through to what lies before it (whole numbers, so every sum is exact)."""
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randint(-4, 5, s, generator=g).float().cuda() for s in ((16, 32), (32, 24)))
    d = rr.Dropout(0.5, 3)
    w.requires_grad_()
    rr.dropout(x @ w, d).square().sum().backward()
    y = rr.dropout((x @ w).detach(), d)
    assert torch.equal(w.grad, x.t() @ rr.dropout(2 * y, d))


def test_dropout_on_another_stream_records_its_gradient(rr):
    side, d = torch.cuda.Stream(), rr.Dropout(0.5, 3)
    x, dy = draw(64, 65, 1, F32).requires_grad_(), draw(64, 65, 2, F32)
    side.wait_stream(torch.cuda.current_stream())
    y = rr.dropout(x, d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    y.backward(dy)
    assert torch.equal(x.grad, rr.dropout(dy, d))


def test_a_given_output_records_no_gradient(rr):
    """out= is refused where a gradient would be lost, and taken where none is recorded."""
    d = rr.Dropout(0.5, 3)
    x, r = draw(4, 64, 1, F32), draw(4, 64, 2, F32)
    learns = x.clone().requires_grad_()
    for args in (dict(x=learns, out=torch.empty_like(x)), dict(x=x, residual=learns, out=torch.empty_like(x))):
        with pytest.raises(ValueError, match="gradient"):
            rr.dropout(drop=d, **args)
        with torch.no_grad():
            assert rr.dropout(drop=d, **args) is args["out"]
    out = torch.empty_like(x)
    rr.dropout(x, d, residual=r, out=out)
    assert torch.equal(out, rr.dropout(x, d, residual=r)) and not out.requires_grad


def test_product_passes_the_residuals_gradient_on(rr):
    """The 4-bit operands hold no gradient; the residual's is dy."""
    a, b = rr.mx4_quantize(draw(40, 64, 1)), rr.mx4_quantize(draw(50, 64, 2))
    r, dy, d = draw(40, 50, 3).requires_grad_(), draw(40, 50, 4), rr.Dropout(0.2, 1)
    want = rr.mx4_matmul(a, b, residual=r.detach(), dropout=d)
    for stream in (None, torch.cuda.current_stream()):
        y = rr.mx4_matmul(a, b, residual=r, dropout=d, stream=stream)
        assert torch.equal(y.detach(), want)
        y.backward(dy)
        assert torch.equal(r.grad, dy)
        r.grad = None
    with pytest.raises(ValueError, match="gradient"):
        rr.mx4_matmul(a, b, residual=r, out=torch.empty_like(want))
    with torch.no_grad():
        out = torch.empty_like(want)
        assert rr.mx4_matmul(a, b, residual=r, dropout=d, out=out) is out and torch.equal(out, want)
