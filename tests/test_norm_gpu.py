"""Layer norm and its backward pass against the definition in 64 bits.

Tolerances.  u = 2^-24.  A sum over a row is a tree of depth D (a thread's
elements, five shuffles, the warps): its error is at most D u times the sum of
magnitudes.  Forward, with s = sqrt(var + eps): the mean is off by m = (D + 1) u
mean|x|; x - mean by m + u |x - mean|; the variance, relative, by (D + 4) u + 2 m
/ s; rstd by half of that and 2 u; y by |w| (m + u |d|) / s + |w h| (rstd's + 2 u)
+ u |y|, then half a step of its format.  Backward, with mean and rstd given: h
is off by 3 u |h| (its subtraction and product; where x - mean cancels, the
subtraction is exact), g by u |g|, the sums by D u of their magnitudes and their
terms' errors, and each of the four operations behind them by u."""
import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
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


def draw(shape, seed, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def depth(cols):
    """Additions on the way of one element of a row's sum, at most."""
    return 32 + 5 + 32 + cols // 512


def check_forward(y, mean, rstd, x, w, b, eps):
    want, m, r, h = ref.norm(x, w, b, eps)
    D, xd = depth(x.shape[-1]), x.double()
    off_m = (D + 1) * U * xd.abs().mean(-1, keepdim=True)
    r = r.unsqueeze(-1)
    off_r = 0.5 * ((D + 4) * U + 2 * off_m * r) + 2 * U
    wa = torch.ones_like(h) if w is None else w.double().abs()
    bound = wa * (off_m * r + U * h.abs()) + wa * h.abs() * (off_r + 2 * U) + U * want.abs()
    bound = bound * 1.01 + ref.half_step(y.dtype) * (want.abs() + bound) + torch.finfo(y.dtype).tiny * ref.half_step(y.dtype) * 2
    assert ((y.double() - want).abs() <= bound).all()
    if mean is not None:
        assert ((mean.double() - m).abs() <= off_m.squeeze(-1) * 1.01).all()
        assert ((rstd.double() - r.squeeze(-1)).abs() <= (off_r * r).squeeze(-1) * 1.01).all()


def check_backward(got, dy, x, mean, rstd, w):
    dx, dw, db = got
    want_x, want_w, want_b = ref.norm_grad(dy, x, mean, rstd, w)
    D, n = depth(x.shape[-1]) + 8, x.shape[-1]
    h = (x.double() - mean.double().unsqueeze(-1)) * rstd.double().unsqueeze(-1)
    d = dy.double()
    g = d if w is None else d * w.double()
    off_1 = (D + 1) * U * g.abs().mean(-1, keepdim=True)
    off_2 = (D + 6) * U * (g * h).abs().mean(-1, keepdim=True)
    s1, s2 = g.mean(-1, keepdim=True).abs(), (g * h).mean(-1, keepdim=True).abs()
    bound = rstd.double().unsqueeze(-1) * (off_1 + h.abs() * off_2 + 6 * U * (g.abs() + s1 + h.abs() * s2))
    if dx is not None:
        top = torch.finfo(dx.dtype)
        assert ((dx.double() - want_x).abs() <= bound * 1.01 + top.eps / 2 * (want_x.abs() + bound) + top.tiny * top.eps).all()
    rows = x.numel() // max(n, 1)
    D = rows // 64 + 80
    axes = tuple(range(d.dim() - 1))
    for out, want, size in ((dw, want_w, (d * h).abs().sum(axes)), (db, want_b, d.abs().sum(axes))):
        if out is not None:
            top = torch.finfo(out.dtype)
            bound = (D + 4) * U * size * 1.01
            assert ((out.double() - want).abs() <= bound + top.eps / 2 * (want.abs() + bound) + top.tiny * top.eps).all()


# every path of the launchers: groups of 16 bytes on 32 to 1024 threads, single elements, rows longer than registers
SHAPES = [(1, 1), (3, 8), (1, 4096), (37, 256), (300, 33), (7, 248), (61, 512), (130, 777), (9, 1000), (1000, 1024),
          (70, 1999), (33, 2048), (700, 4096), (12, 4095), (5, 8192), (6, 8191), (3, 16384), (4, 10001), (2, 32768),
          (3, 40000), (2, 70003), (5003, 96)]


@pytest.mark.parametrize("dtype,wtype", [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_both_passes(rr, rows, cols, dtype, wtype):
    x, dy = draw((rows, cols), 1, dtype, 2.0, 0.7), draw((rows, cols), 2, dtype)
    w, b = draw(cols, 3, wtype, 0.3, 1.0), draw(cols, 4, wtype)
    y, mean, rstd = rr.layer_norm_forward(x, w, b)
    check_forward(y, mean, rstd, x, w, b, 1e-5)
    check_backward(rr.layer_norm_backward(dy, x, mean, rstd, w), dy, x, mean, rstd, w)
    assert rr.device_status() == 0


@pytest.mark.parametrize("cols", [96, 777, 20000])
def test_without_weights(rr, cols):
    x, dy = draw((50, cols), 1, BF16), draw((50, cols), 2, BF16)
    y, mean, rstd = rr.layer_norm_forward(x)
    check_forward(y, mean, rstd, x, None, None, 1e-5)
    w = draw(cols, 3, F32)
    check_forward(rr.layer_norm(x, w), None, None, x, w, None, 1e-5)
    check_forward(rr.layer_norm(x, None, w, eps=0.5), None, None, x, None, w, 0.5)
    dx, dw, db = rr.layer_norm_backward(dy, x, mean, rstd, wdtype=F32)
    assert dw.dtype == F32
    check_backward((dx, dw, db), dy, x, mean, rstd, None)


@pytest.mark.parametrize("cols", [96, 777, 20000])
def test_a_large_mean_keeps_the_variance(rr, cols):
    """Where the mean is a thousand times the spread, the squares' difference would leave nothing of it."""
    x = draw((40, cols), 1, F32, 1.0, 1000.0)
    y, mean, rstd = rr.layer_norm_forward(x, eps=0.0)
    check_forward(y, mean, rstd, x, None, None, 0.0)


def test_constant_and_tiny_rows(rr):
    x = torch.full((3, 640), 2.5, device="cuda")
    x[1] = 0
    y, mean, rstd = rr.layer_norm_forward(x, eps=1e-5)
    assert (y == 0).all() and mean.tolist() == [2.5, 0, 2.5]
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    one = rr.layer_norm(torch.tensor([[3.0], [4.0]], device="cuda"), bias=torch.tensor([7.0], device="cuda"))
    assert one.tolist() == [[7.0], [7.0]]


def test_not_finite_rows_stay_alone(rr):
    x = draw((6, 1024), 1, BF16)
    clean = rr.layer_norm(x)
    x[1, 5], x[4, 7] = float("inf"), float("nan")
    y = rr.layer_norm(x)
    assert y[[1, 4]].isnan().all()
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols,pad,at", [(40, 96, 32, 16), (40, 96, 7, 3), (33, 1001, 23, 8), (5, 4096, 64, 0),
                                              (3, 33000, 8, 8)])
def test_strides_guards_and_in_place(rr, rows, cols, pad, at, dtype):
    """Rows of a wider array, on the 16-byte grid and off it; nothing beside them is written; in place gives the same bits."""
    whole = torch.full((rows, cols + pad), 7.0, dtype=dtype, device="cuda")
    v = whole[:, at:at + cols]
    x, dy, w, b = draw((rows, cols), 1, dtype), draw((rows, cols), 2, dtype), draw(cols, 3, dtype), draw(cols, 4, dtype)
    v.copy_(x)
    y, mean, rstd = rr.layer_norm_forward(v, w, b)
    check_forward(y, mean, rstd, x, w, b, 1e-5)
    got = rr.layer_norm_backward(dy, v, mean, rstd, w)
    check_backward(got, dy, x, mean, rstd, w)
    rr.layer_norm(v, w, b, out=v)
    assert torch.equal(v, y)
    assert (whole[:, :at] == 7).all() and (whole[:, at + cols:] == 7).all()
    v.copy_(dy)
    check_backward(rr.layer_norm_backward(v, x, mean, rstd, w), dy, x, mean, rstd, w)


@pytest.mark.parametrize("cols", [96, 1001, 4096, 20000])
def test_gradient_in_place_through_the_c_abi(rr, cols):
    x, dy, w = draw((21, cols), 1, BF16), draw((21, cols), 2, BF16), draw(cols, 3, BF16)
    _, mean, rstd = rr.layer_norm_forward(x, w)
    dx, dw, db = rr.layer_norm_backward(dy, x, mean, rstd, w)
    need = rr.lib().ring_layer_norm_workspace(21, cols)
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    for inout in (0, 1):
        a, b = x.clone(), dy.clone()
        out = (a, b)[inout]
        sw, sb = torch.empty_like(w), torch.empty_like(w)
        st = rr.lib().ring_layer_norm_backward(b.data_ptr(), cols, a.data_ptr(), cols, w.data_ptr(), 2, mean.data_ptr(),
                                               rstd.data_ptr(), out.data_ptr(), cols, sw.data_ptr(), sb.data_ptr(), 21, cols, 2,
                                               space.data_ptr(), need, torch.cuda.current_stream().cuda_stream or None)
        assert st == 0
        assert torch.equal(out, dx) and torch.equal(sw, dw) and torch.equal(sb, db)


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True), (False, True, True)])
@pytest.mark.parametrize("cols", [96, 1001, 20000])
def test_parts_of_the_gradient(rr, cols, want):
    x, dy, w = draw((70, cols), 1, F16), draw((70, cols), 2, F16), draw(cols, 3, F16)
    _, mean, rstd = rr.layer_norm_forward(x, w)
    full = rr.layer_norm_backward(dy, x, mean, rstd, w)
    for g, f, k in zip(rr.layer_norm_backward(dy, x, mean, rstd, w, *want), full, want):
        assert torch.equal(g, f) if k else g is None


def test_no_rows_and_no_columns(rr):
    w = draw(40, 3, F32)
    x = torch.empty((0, 40), device="cuda")
    y, mean, rstd = rr.layer_norm_forward(x, w)
    dx, dw, db = rr.layer_norm_backward(x, x, mean, rstd, w)
    assert y.shape == dx.shape == (0, 40) and (dw == 0).all() and (db == 0).all()
    x = torch.empty((5, 0), device="cuda")
    y, mean, rstd = rr.layer_norm_forward(x)
    assert y.shape == (5, 0) and rr.layer_norm_backward(x, x, mean, rstd)[1].shape == (0,)


def test_same_bits_every_time(rr):
    x, dy, w = draw((3001, 1024), 1, BF16), draw((3001, 1024), 2, BF16), draw(1024, 3, F32)
    _, mean, rstd = rr.layer_norm_forward(x, w)
    first = rr.layer_norm_backward(dy, x, mean, rstd, w)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(rr.layer_norm_backward(dy, x, mean, rstd, w), first))


def test_past_four_billion_elements(rr):
    """Rows beyond element 2^32 of x and y."""
    rows, cols = (1 << 32) // 4096 + 3, 4096
    x = torch.empty((rows, cols), dtype=BF16, device="cuda")
    x.fill_(1.0)
    x[-2:] = draw((2, cols), 1, BF16)
    dy = torch.zeros((rows, cols), dtype=BF16, device="cuda")
    dy[-2:] = draw((2, cols), 2, BF16)
    y, mean, rstd = rr.layer_norm_forward(x)
    check_forward(y[-2:], mean[-2:], rstd[-2:], x[-2:], None, None, 1e-5)
    assert (y[0] == 0).all() and (y[rows // 2] == 0).all()
    got = rr.layer_norm_backward(dy, x, mean, rstd, wdtype=F32)
    check_backward((got[0][-2:],) + got[1:], dy[-2:], x[-2:], mean[-2:], rstd[-2:], None)
    del x, y, dy, got
    torch.cuda.empty_cache()


# ------------------------------------------------------------------- autograd


@pytest.mark.parametrize("need", [(1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)])
def test_autograd(rr, need):
    x, w, b, dy = draw((4, 6, 160), 1), draw(160, 2), draw(160, 3), draw((4, 6, 160), 4)
    for t, k in zip((x, w, b), need):
        t.requires_grad_(bool(k))
    y = rr.layer_norm(x, w, b)
    y.backward(dy)
    with torch.no_grad():
        y2, mean, rstd = rr.layer_norm_forward(x, w, b)
        want = rr.layer_norm_backward(dy, x, mean, rstd, w)
    assert torch.equal(y, y2)
    for t, g, k in zip((x, w, b), want, need):
        assert torch.equal(t.grad, g) if k else t.grad is None


def test_gradient_against_differences(rr):
    """Central differences of the kernel's own output in binary32: off by h^2 / 6 times the third derivative, and by the
    output's rounding (about 10 u |y| an element, 24 * 160 of them in quadrature) over h."""
    x, w, b, dy = draw((24, 160), 1), draw(160, 2), draw(160, 3), draw((24, 160), 4)
    for t in (x, w, b):
        t.requires_grad_()
    rr.layer_norm(x, w, b).backward(dy)
    h = 2.0 ** -6
    for t, seed in ((x, 5), (w, 6), (b, 7)):
        v = draw(tuple(t.shape), seed)
        v /= v.norm()
        with torch.no_grad():
            args = lambda s: [u + s * v if u is t else u for u in (x, w, b)]
            up, down = (rr.layer_norm(*args(s)).double() for s in (h, -h))
        slope = ((up - down) * dy.double()).sum().item() / (2 * h)
        noise = 20 * U * (24 * 160) ** 0.5 * 10 / (2 * h)
        # third derivative along a unit direction of rows with a spread of one: at most 15 |v|^3 |w| |dy|, all below 5
        assert abs(slope - (t.grad.double() * v.double()).sum().item()) <= noise + h * h / 6 * 15 * 25


def test_expanded_gradient(rr):
    """y.sum() hands back a gradient whose strides are zero."""
    x = draw((30, 96), 1).requires_grad_()
    w = draw(96, 2).requires_grad_()
    rr.layer_norm(x, w).sum().backward()
    ones = torch.ones((30, 96), device="cuda")
    with torch.no_grad():
        _, mean, rstd = rr.layer_norm_forward(x, w)
        want = rr.layer_norm_backward(ones, x, mean, rstd, w)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])


def test_refusals(rr):
    x, w = draw((6, 96), 1, BF16), draw(96, 2, BF16)
    bad = [lambda: rr.layer_norm(x.cpu()), lambda: rr.layer_norm(x, w[:95]), lambda: rr.layer_norm(x, w.half()),
           lambda: rr.layer_norm(x, w, w.float()), lambda: rr.layer_norm(x.t()), lambda: rr.layer_norm(x.double()),
           lambda: rr.layer_norm(x, out=x[:5]), lambda: rr.layer_norm(x, out=x.float()),
           lambda: rr.layer_norm(x.clone().requires_grad_(), out=x), lambda: rr.layer_norm_forward(x.clone().requires_grad_()),
           lambda: rr.layer_norm(torch.tensor(1.0, device="cuda")), lambda: rr.layer_norm(x, w.cpu())]
    y, mean, rstd = rr.layer_norm_forward(x, w)
    bad += [lambda: rr.layer_norm_backward(y[:5], x, mean, rstd, w), lambda: rr.layer_norm_backward(y, x, mean[:5], rstd, w),
            lambda: rr.layer_norm_backward(y, x, mean, rstd.double(), w), lambda: rr.layer_norm_backward(y.float(), x, mean, rstd, w),
            lambda: rr.layer_norm_backward(y, x, mean, rstd, wdtype=F16)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(rr.RingError):
            rr.layer_norm(x, eps=eps)


def test_another_stream_and_a_graph(rr):
    x, dy, w = draw((200, 1024), 1, BF16), draw((200, 1024), 2, BF16), draw(1024, 3, BF16)
    y, mean, rstd = rr.layer_norm_forward(x, w)
    want = (y,) + rr.layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, mean2, rstd2 = rr.layer_norm_forward(x, w, stream=side)
    got = (y2,) + rr.layer_norm_backward(dy, x, mean2, rstd2, w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    xs, ds = torch.zeros_like(x), torch.zeros_like(dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, mean3, rstd3 = rr.layer_norm_forward(xs, w)
        got = (y3,) + rr.layer_norm_backward(ds, xs, mean3, rstd3, w)
    for k in range(2):
        xs.copy_(x), ds.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        xs.zero_(), ds.zero_()
        graph.replay()
