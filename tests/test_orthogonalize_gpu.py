"""The orthogonalised update against the definition in 64 bits.

Tolerances.  X, S and b S + c S^2 are rounded to binary16, half a step of which is
2^-11.  The reference computes the steps in 64 bits twice: as they are, and with
the same three roundings.  The kernel's sums in binary32 differ from 64 bits by
far less than binary16's half step (2^-22 (K / 16 + 4) of the sum of magnitudes),
so its error is another draw of the same roundings: in the Frobenius norm it is
held to twice what they do to the reference, and the rounding of the result."""
import pytest
import torch

import training_reference as ref

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


def draw(shape, seed, dtype=F32, scale=1e-2):
    """A few strong directions and noise."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    b = shape[:-2]
    return ((r(*b, shape[-2], 16) @ r(*b, 16, shape[-1]) / 4 + 0.3 * r(*shape)) * scale).to(dtype)


def norms(t):
    return torch.linalg.matrix_norm(t.double())


def check(y, g, steps=5, eps=1e-7):
    want, held = ref.orthogonal(g, steps, eps), ref.orthogonal(g, steps, eps, held=True)
    # (below: a result that is exact but for its own rounding, as of one row)
    bound = 2 * norms(held - want) + (ref.half_step(y.dtype) + 2.0 ** -18) * norms(want)
    off = norms(y.double() - want)
    assert y.isfinite().all() and (off <= bound).all(), (off, bound)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (16, 16), (32, 100), (100, 32), (127, 129), (128, 128), (128, 512), (640, 130),
          (777, 1537), (1537, 777), (1000, 1000), (34, 4240), (128, 129), (100, 300), (640, 90), (128, 900), (33, 1024), (1025, 128), (77, 2048), (2040, 65), (64, 2049), (2048, 2048), (1100, 2600), (2600, 1100), (4100, 260), (2300, 2400), (2400, 2310), (100, 8000), (8000, 100)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,out", [(F32, BF16), (BF16, None), (F16, F32)])
def test_matrices(rr, rows, cols, dtype, out):
    g = draw((rows, cols), 1, dtype)
    y = rr.orthogonalize(g, dtype=out)
    torch.cuda.synchronize()
    assert rr.device_status() == 0
    assert y.dtype == (out or dtype)
    check(y, g)


@pytest.mark.parametrize("shape", [(3, 40, 70), (8, 128, 512), (2, 300, 130), (5, 600, 600), (0, 4, 5), (3, 1030, 1040)])
def test_batches(rr, shape):
    g = draw(shape, 2)
    y = rr.orthogonalize(g, dtype=BF16)
    if shape[0]:
        check(y, g)
        for k in range(shape[0]):
            assert torch.equal(rr.orthogonalize(g[k], dtype=BF16), y[k]) or shape[0] * shape[1] > 2000
    assert y.shape == shape


@pytest.mark.parametrize("steps", [1, 2, 3, 10])
def test_steps(rr, steps):
    g = draw((200, 333), 3)
    check(rr.orthogonalize(g, steps=steps), g, steps)


def test_singular_values_come_near_one(rr):
    """A matrix with known singular vectors, its values 1 .. 0.05: each goes through the scalar polynomial."""
    q = lambda n, k, seed: torch.linalg.qr(torch.randn((n, k), generator=torch.Generator().manual_seed(seed)).double())[0].cuda()
    u, v, s = q(300, 64, 1), q(400, 64, 2), torch.linspace(1, 0.05, 64, dtype=torch.float64, device="cuda")
    y = rr.orthogonalize((u * s @ v.T).float())
    a, b, c = ref.QUINTIC
    t = s / s.norm()
    for _ in range(5):
        t = a * t + b * t ** 3 + c * t ** 5
    got = u.T @ y.double() @ v
    assert (got.diagonal() - t).abs().max() < 0.02 and 0.6 < got.diagonal().min() and got.diagonal().max() < 1.25
    assert (got - got.diagonal().diag()).abs().max() < 0.02


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_any_scale(rr, dtype, scale):
    """The norm neither overflows nor vanishes; eps is small beside it only if the matrix is not."""
    g = draw((60, 90), 4, dtype, scale)
    assert g.isfinite().all()
    check(rr.orthogonalize(g, eps=0.0, dtype=F32), g, eps=0.0)
    check(rr.orthogonalize(g, dtype=F32), g)


def test_zeros_and_no_numbers(rr):
    g = draw((4, 60, 90), 5)
    clean = rr.orthogonalize(g)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    g[3, 1, 1] = float("inf")
    y = rr.orthogonalize(g)
    assert torch.equal(y[0], clean[0]) and (y[1] == 0).all() and y[2].isnan().all() and not y[3].isfinite().any()


@pytest.mark.parametrize("pad,at", [(6, 0), (16, 16), (3, 1)])
@pytest.mark.parametrize("rows,cols", [(60, 90), (90, 60), (300, 1000), (40, 1400), (700, 40)])
def test_strides_guards_and_in_place(rr, rows, cols, pad, at):
    g = draw((2, rows, cols), 6, BF16)
    want = rr.orthogonalize(g)
    whole = torch.full((2, rows + 2, cols + pad + at), 7.0, dtype=BF16, device="cuda")
    v = whole[:, 1:1 + rows, at:at + cols]
    v.copy_(g)
    assert torch.equal(rr.orthogonalize(v), want)
    rr.orthogonalize(v, out=v)
    assert torch.equal(v, want)
    whole[:, 1:1 + rows, at:at + cols] = 7
    assert (whole == 7).all()


def test_nothing_past_the_workspace(rr):
    L = rr.lib()
    for shape in ((1, 60, 90), (3, 777, 513), (2, 128, 1500)):
        g = draw(shape, 7)
        want = rr.orthogonalize(g)
        need = L.ring_orthogonalize_workspace(*shape)
        out = torch.full(shape, 7.0, device="cuda")
        space = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")  # (binary16 NaN everywhere)
        _, m, n = shape
        st = L.ring_orthogonalize(g.data_ptr(), n, m * n, 0, out.data_ptr(), n, m * n, 0, *shape, 5, 1e-7, space.data_ptr(), need,
                                  torch.cuda.current_stream().cuda_stream or None)
        assert st == 0 and torch.equal(out, want) and (space[need:] == 0xFF).all()


def test_past_four_billion_elements(rr):
    """Matrices of a batch beyond element 2^32 of g, of the iterates and of the output."""
    batch, n = 260, 4096
    g = torch.empty((batch, n, n), dtype=BF16, device="cuda")
    for k in range(batch):
        g[k] = draw((n, n), 12 + k % 3, BF16)
    y = rr.orthogonalize(g, steps=2)
    for k in (0, batch - 1):
        check(y[k], g[k], 2)
    assert torch.equal(y[batch - 3], y[batch - 6])  # (the same matrix)
    del g, y
    torch.cuda.empty_cache()


def test_same_bits_every_time(rr):
    g = draw((1100, 1300), 8, BF16)
    first = rr.orthogonalize(g)
    assert all(torch.equal(rr.orthogonalize(g), first) for _ in range(5))


def test_empty(rr):
    for shape in ((0, 5), (5, 0), (2, 0, 3)):
        assert rr.orthogonalize(torch.empty(shape, device="cuda")).shape == shape


def test_refusals(rr):
    g = draw((20, 30), 9)
    for call in (lambda: rr.orthogonalize(g.cpu()), lambda: rr.orthogonalize(g.t()), lambda: rr.orthogonalize(g.double()),
                 lambda: rr.orthogonalize(g[0]), lambda: rr.orthogonalize(g, out=g[:10]), lambda: rr.orthogonalize(g, dtype=torch.int32),
                 lambda: rr.orthogonalize(g, dtype=F16, out=g), lambda: rr.orthogonalize(g.clone().requires_grad_()),
                 lambda: rr.orthogonalize(g.expand(4, 20, 30))):
        with pytest.raises(ValueError):
            call()
    for how in (dict(steps=0), dict(steps=1001), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(rr.RingError):
            rr.orthogonalize(g, **how)
    with torch.no_grad():
        rr.orthogonalize(g.clone().requires_grad_())


def test_another_stream_and_graphs(rr):
    g, g2 = draw((300, 500), 10), draw((300, 500), 11)
    want, want2 = rr.orthogonalize(g), rr.orthogonalize(g2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = rr.orthogonalize(g, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    held = g.clone()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = rr.orthogonalize(held)
        graphs.append((graph, out))
    for x, expect in ((g2, want2), (g, want)):
        held.copy_(x)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, expect) for _, out in graphs)
