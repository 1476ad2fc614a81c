"""What the differentiable 4-bit layer keeps for its backward pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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
