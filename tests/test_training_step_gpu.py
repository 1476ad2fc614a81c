"""The operators of a training step together: norm, 4-bit layer, norm, loss, the ranks' sum and the orthogonalised step, as
the example runs them; in a graph; on two streams at once."""
import importlib.util
import os

import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import ring_allreduce_reducescatter_gb300 as mod

    torch.cuda.set_device(0)
    return mod


@pytest.fixture(scope="module")
def example(rr):
    spec = importlib.util.spec_from_file_location("muon_data_parallel", os.path.join(ROOT, "examples", "muon_data_parallel.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def batch(tokens, vocabulary, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    here = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
    there = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
    there[:5] = -100
    return here, there


def test_the_example_runs(rr, example):
    losses = example.train(ranks=2, tokens=96, features=64, vocabulary=130, steps=3)
    assert len(losses) == 3 and all(0 < x < 100 for x in losses)
    assert rr.device_status() == 0


def test_gradients_of_the_example(rr, example):
    """Each trained parameter's gradient against 64 bits, through the operators' own intermediate values: the output matrix
    and the last norm, whose gradients do not pass the 4-bit layer."""
    tokens, features, vocabulary = 200, 96, 333
    p = example.parameters(features, vocabulary)
    p["norm2"] = 1 + 0.1 * torch.randn(features, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8))
    here, there = batch(tokens, vocabulary)
    _, got = example.gradients(p, here, there, seed=5, subsequence=9)
    x = p["embedding"][here]
    h = rr.mx4_linear(rr.layer_norm(x, p["norm1"], p["bias1"]), p["layer"], residual=x, seed=5, subsequence=9)
    y, mean, rstd = rr.layer_norm_forward(h, p["norm2"])
    grad = torch.tensor(1.0 / int((there != -100).sum()), device="cuda")
    e = ref.cross_entropy_grad(grad, y.double() @ p["output"].double().t(), there, -100)
    off = ref.half_step(BF16)
    # half a step for e's rounding and one for the result's, in the Frobenius norm, and binary32's sums
    assert (got["output"].double() - e.t() @ y.double()).norm() <= 2 * off * (e.t() @ y.double()).norm()
    dy = rr.linear_cross_entropy_backward(grad, y, p["output"], there,
                                          rr.linear_cross_entropy_forward(y, p["output"], there)[1])[0]
    dh, dw, _ = ref.norm_grad(dy, h, mean, rstd, p["norm2"])
    size = (dy.double().abs() * ((h.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs()).sum(0)
    assert ((got["norm2"].double() - dw).abs() <= (tokens + 80) * ref.U * size).all()
    # what passes the 4-bit layer: the layer's own gradient of the same dh
    _, dh_own = rr.layer_norm_forward(h, p["norm2"])[0], rr.layer_norm_backward(dy, h, mean, rstd, p["norm2"])[0]
    assert (dh_own.double() - dh).norm() <= 2 * off * dh.norm()
    w = p["layer"].detach().requires_grad_()
    n = rr.layer_norm(x, p["norm1"], p["bias1"]).detach().requires_grad_()
    rr.mx4_linear(n, w, residual=x, seed=5, subsequence=9).backward(dh_own)
    assert torch.equal(got["layer"], w.grad)
    _, m1, r1 = rr.layer_norm_forward(x, p["norm1"], p["bias1"])
    want = rr.layer_norm_backward(n.grad, x, m1, r1, p["norm1"])
    assert torch.equal(got["norm1"], want[1]) and torch.equal(got["bias1"], want[2])


def test_a_step_in_a_graph(rr, example):
    """Forward, backward, the ranks' sum and the update captured once and replayed over new tokens: the eager bits."""
    tokens, features, vocabulary, ranks = 160, 128, 500, 2
    p = example.parameters(features, vocabulary)

    def step(batches):
        grads = [example.gradients(p, here, there, drop=rr.Dropout(0.1, 3, 5 + r), seed=3, subsequence=20 + 4 * r)
                 for r, (here, there) in enumerate(batches)]
        sums = {k: rr.allreduce([g[k].float().reshape(-1) for _, g in grads])[0].view(p[k].shape) for k in example.TRAINED}
        return [l for l, _ in grads] + [sums[k] for k in example.TRAINED] + [rr.orthogonalize(sums["layer"], dtype=BF16)]

    old, new = ([batch(tokens, vocabulary, s + r) for r in range(ranks)] for s in (10, 20))
    want_old, want_new = [t.clone() for t in step(old)], [t.clone() for t in step(new)]
    held = [(a.clone(), b.clone()) for a, b in old]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(held)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    for batches, want in ((new, want_new), (old, want_old), (new, want_new)):
        for (a, b), (x, y) in zip(held, batches):
            a.copy_(x), b.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert rr.device_status() == 0


def test_two_streams_at_once(rr):
    """Calls whose workspaces live at the same time, on two streams, over and over."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((300, 512), generator=g, device="cuda").to(BF16)
    w = (torch.randn((4000, 512), generator=g, device="cuda") * 0.05).to(BF16)
    target = torch.randint(0, 4000, (300,), generator=g, device="cuda")
    grad = torch.full((), 0.5, device="cuda")
    weight = torch.randn(512, generator=g, device="cuda")

    def calls(stream=None):
        how = {} if stream is None else {"stream": stream}
        y, mean, rstd = rr.layer_norm_forward(x, weight, **how)
        loss, lse = rr.linear_cross_entropy_forward(y, w, target, **how)
        dx, dw = rr.linear_cross_entropy_backward(grad, y, w, target, lse, **how)
        d = rr.layer_norm_backward(dx, x, mean, rstd, weight, **how)
        return [y, loss, dx, dw, *d, rr.orthogonalize(dw, **how), rr.orthogonalize(dx[:100], **how)]

    want = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [calls(s) for s in streams]
        torch.cuda.synchronize()
        for out in got:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_saved_tensors_and_a_second_backward_pass(rr):
    """What the norm and the loss keep is seen by saved-tensor hooks; a second backward pass needs a graph that was asked to
    stay, and gives the same gradients again."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((60, 96), generator=g, device="cuda").to(BF16).requires_grad_()
    w = (torch.randn((200, 96), generator=g, device="cuda") * 0.1).to(BF16).requires_grad_()
    target = torch.randint(0, 200, (60,), generator=g, device="cuda")
    loss = rr.linear_cross_entropy(rr.layer_norm(x), w, target)
    loss.backward(retain_graph=True)
    once = x.grad.clone(), w.grad.clone()
    loss.backward()
    assert torch.equal(x.grad, 2 * once[0]) and torch.equal(w.grad, 2 * once[1])
    with pytest.raises(RuntimeError, match="second time"):
        loss.backward()
    x.grad = w.grad = None
    with torch.autograd.graph.save_on_cpu():
        loss = rr.linear_cross_entropy(rr.layer_norm(x), w, target)
    loss.backward()
    assert torch.equal(x.grad, once[0]) and torch.equal(w.grad, once[1])
    for call in (lambda: torch.autograd.grad(rr.linear_cross_entropy(rr.layer_norm(x), w, target), x, create_graph=True)[0].sum(),):
        with pytest.raises(RuntimeError):
            call().backward()


def test_changed_in_place_after_the_forward_pass(rr):
    x = torch.randn((60, 96), device="cuda").requires_grad_()
    a = x * 1
    y = rr.layer_norm(a)
    a.add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
