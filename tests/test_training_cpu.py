"""CPU tests of the operators of a training step: the references against differences and hand-worked values, and the C
ABI's refusals (no kernel is launched)."""
import pytest
import torch

import training_reference as ref

OK, EINVAL, EUNSUP, EALIAS, ECUDA = range(5)
F32, F16, BF16 = 0, 1, 2
BASE = 0x7F0000000000  # never dereferenced
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    from ring_allreduce_reducescatter_gb300 import _build

    _build.build()
    import ring_allreduce_reducescatter_gb300 as rr

    return rr.lib()


def slope(f, v, h=1e-5):
    return (f(h * v) - f(-h * v)) / (2 * h)


# ------------------------------------------------------------------ layer norm


def test_norm_by_hand():
    y, mean, rstd, _ = ref.norm(torch.tensor([[1.0, 3.0], [5.0, 5.0]]), torch.tensor([2.0, 1.0]), torch.tensor([0.5, 0.0]), 0.0)
    assert y[0].tolist() == [-1.5, 1.0] and mean.tolist() == [2.0, 5.0] and rstd[0] == 1.0


def test_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    x, w, b, dy = (torch.randn(s, generator=g).double() for s in ((7, 12), (12,), (12,), (7, 12)))
    _, mean, rstd, _ = ref.norm(x, w, b, 1e-3)
    dx, dw, db = ref.norm_grad(dy, x, mean, rstd, w)
    for grad, at in ((dx, 0), (dw, 1), (db, 2)):
        v = torch.randn(grad.shape, generator=g).double()

        def loss(step):
            args = [x, w, b]
            args[at] = args[at] + step
            return (ref.norm(*args, 1e-3)[0] * dy).sum().item()

        assert abs(slope(loss, v) - (grad * v).sum().item()) < 1e-6


def test_layer_norm_refusals(L):
    x, out, w, b, m, r = (BASE + k * MB for k in range(6))

    def call(x=x, ldx=96, w=w, b=b, wt=F32, eps=1e-5, out=out, ldo=96, m=m, r=r, rows=64, cols=96, dtype=BF16):
        return L.ring_layer_norm(x, ldx, w, b, wt, eps, out, ldo, m, r, rows, cols, dtype, None)

    assert call() == ECUDA  # valid: fails only for want of a GPU
    assert call(w=None, b=None, m=None, r=None) == ECUDA and call(out=x) == ECUDA and call(wt=BF16) == ECUDA
    assert call(x=x, out=x + 192, ldx=200, ldo=200) == ECUDA  # beside one another
    assert call(wt=F16) == EINVAL and call(dtype=3) == EINVAL and call(wt=7) == EINVAL
    assert call(eps=-1.0) == EINVAL and call(eps=float("nan")) == EINVAL and call(eps=float("inf")) == EINVAL
    assert call(x=None) == EINVAL and call(x=x + 1) == EINVAL and call(ldx=95) == EINVAL and call(ldo=95) == EINVAL
    assert call(out=None) == EINVAL and call(w=w + 2) == EINVAL and call(m=m + 2) == EINVAL
    assert call(rows=1 << 31) == EINVAL and call(cols=1 << 31) == EINVAL
    assert call(out=x + 64) == EALIAS and call(out=x, ldo=100) == EALIAS and call(m=x) == EALIAS and call(r=m) == EALIAS
    assert call(out=w) == EALIAS and call(m=b) == EALIAS and call(r=out) == EALIAS
    assert call(rows=0) == OK and call(cols=0) == OK


def test_layer_norm_backward_refusals(L):
    dy, x, w, m, r, dx, dw, db, ws = (BASE + k * MB for k in range(9))
    need = L.ring_layer_norm_workspace(64, 96)
    assert need == 64 * 2 * 96 * 4 and L.ring_layer_norm_workspace(0, 96) == 0

    def call(dy=dy, ldy=96, x=x, ldx=96, w=w, wt=F32, m=m, r=r, dx=dx, ldd=96, dw=dw, db=db, rows=64, cols=96, dtype=BF16,
             ws=ws, wb=need):
        return L.ring_layer_norm_backward(dy, ldy, x, ldx, w, wt, m, r, dx, ldd, dw, db, rows, cols, dtype, ws, wb, None)

    assert call() == ECUDA and call(dx=dy) == ECUDA and call(dx=x) == ECUDA and call(w=None) == ECUDA
    assert call(dw=None, db=None, ws=None, wb=0) == ECUDA
    assert call(dx=None, dw=None, db=None) == OK and call(cols=0) == OK and call(rows=0, dw=None, db=None) == OK
    assert call(wb=need - 1) == EINVAL and call(ws=None) == EINVAL and call(ws=ws + 8) == EINVAL
    assert call(wt=F16) == EINVAL and call(dtype=9) == EINVAL and call(m=None) == EINVAL and call(r=r + 2) == EINVAL
    assert call(dy=None) == EINVAL and call(ldy=95) == EINVAL and call(ldd=95) == EINVAL and call(dx=dx + 1) == EINVAL
    assert call(rows=1 << 31) == EINVAL
    assert call(dx=dy + 2) == EALIAS and call(dx=x, ldd=97) == EALIAS and call(dw=db) == EALIAS and call(ws=x) == EALIAS
    assert call(dw=dy) == EALIAS and call(dx=w) == EALIAS and call(db=ws) == EALIAS and call(dw=m) == EALIAS


# ------------------------------------------------------- linear cross entropy


def test_cross_entropy_by_hand():
    x, w = torch.eye(2), torch.tensor([[0.0, 1.0], [0.0, 0.0], [0.0, 0.0]])
    loss, lse, _ = ref.cross_entropy(x, w, torch.tensor([2, -100]), -100)
    assert abs(loss[0].item() - torch.log(torch.tensor(3.0, dtype=torch.float64)).item()) < 1e-12 and loss[1] == 0


def test_cross_entropy_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn(s, generator=g).double() for s in ((6, 5), (9, 5)))
    target, grad = torch.tensor([3, -100, 0, 8, 8, 2]), torch.rand(6, generator=g).double()
    e = ref.cross_entropy_grad(grad, x @ w.t(), target, -100)
    for d, at in ((e @ w, 0), (e.t() @ x, 1)):
        v = torch.randn(d.shape, generator=g).double()

        def loss(step):
            args = [x, w]
            args[at] = args[at] + step
            return (ref.cross_entropy(*args, target, -100)[0] * grad).sum().item()

        assert abs(slope(loss, v) - (d * v).sum().item()) < 1e-6


def test_linear_cross_entropy_refusals(L):
    x, w, t, loss, lse, sums, ws = (BASE + k * 16 * MB for k in range(7))
    need = L.ring_linear_cross_entropy_workspace(x, 96, w, 96, 200, 96, 1000)
    assert L.ring_linear_cross_entropy_workspace(x + 2, 96, w, 96, 200, 96, 1000) == need  # (few rows: x is copied in any case)
    assert L.ring_linear_cross_entropy_workspace(x, 96, w, 99, 200, 96, 1000) == need + 1000 * 96 * 2
    assert L.ring_linear_cross_entropy_workspace(x, 96, w, 96, 200, 0, 1000) == 0

    def call(x=x, ldx=96, w=w, ldw=96, t=t, loss=loss, lse=lse, sums=sums, n=200, h=96, v=1000, dtype=BF16, ws=ws, wb=need):
        return L.ring_linear_cross_entropy(x, ldx, w, ldw, t, -100, loss, lse, sums, n, h, v, dtype, ws, wb, None)

    assert call() == ECUDA and call(lse=None, sums=None) == ECUDA and call(dtype=F16) == ECUDA
    assert call(n=0, sums=None) == OK and call(n=0, ws=None, wb=0) == ECUDA
    assert call(dtype=F32) == EUNSUP and call(dtype=5) == EINVAL and call(h=0) == EINVAL and call(v=0) == EINVAL
    assert call(x=None) == EINVAL and call(w=w + 1) == EINVAL and call(t=t + 4) == EINVAL and call(loss=None) == EINVAL
    assert call(ldx=95) == EINVAL and call(ldw=95) == EINVAL and call(wb=need - 1) == EINVAL and call(ws=None) == EINVAL
    assert call(n=1 << 31) == EINVAL and call(v=1 << 31) == EINVAL and call(ws=ws + 8) == EINVAL
    assert call(loss=x) == EALIAS and call(lse=loss) == EALIAS and call(ws=w) == EALIAS and call(sums=t) == EALIAS
    assert call(ws=loss) == EALIAS and call(sums=lse) == EALIAS


def test_linear_cross_entropy_backward_refusals(L):
    g, x, w, t, lse, dx, dw, ws = (BASE + k * 16 * MB for k in range(8))
    need = L.ring_linear_cross_entropy_backward_workspace(x, 96, w, 96, 200, 96, 1000)

    def call(g=g, step=0, x=x, ldx=96, w=w, ldw=96, t=t, lse=lse, dx=dx, lddx=96, dw=dw, lddw=96, n=200, h=96, v=1000,
             dtype=BF16, ws=ws, wb=need):
        return L.ring_linear_cross_entropy_backward(g, step, x, ldx, w, ldw, t, -100, lse, dx, lddx, dw, lddw, n, h, v, dtype, ws,
                                                    wb, None)

    assert call() == ECUDA and call(step=1) == ECUDA and call(dx=None) == ECUDA and call(dw=None) == ECUDA
    assert call(dx=None, dw=None) == OK and call(n=0, dw=None) == OK and call(n=0, ws=None, wb=0) == ECUDA
    assert call(dtype=F32) == EUNSUP and call(dtype=-1) == EINVAL and call(step=2) == EINVAL and call(h=0) == EINVAL
    assert call(g=None) == EINVAL and call(lse=lse + 2) == EINVAL and call(t=None) == EINVAL and call(lddx=90) == EINVAL
    assert call(dw=dw + 1) == EINVAL and call(wb=need - 1) == EINVAL and call(ws=ws + 4) == EINVAL
    assert call(dx=x) == EALIAS and call(dw=w) == EALIAS and call(dx=dw) == EALIAS and call(ws=dx) == EALIAS
    assert call(dw=lse) == EALIAS and call(ws=t) == EALIAS and call(dx=g) == EALIAS


def test_pieces_stay_within_their_memory(L):
    for tokens in (1, 200, 8192, 100_000, 1 << 20):
        for vocabulary in (1, 500, 32000, 131072):
            need = L.ring_linear_cross_entropy_backward_workspace(BASE, 4096, BASE, 4096, tokens, 4096, vocabulary)
            rows = -(-tokens // 128) * 128
            assert need <= max((1 << 28) + 512 * rows, 512 * rows) + tokens * 4096 * 4 + rows * 4096 * 2 * (tokens < 128) + 8 * rows + 4096


# -------------------------------------------------------- orthogonalised update


def test_orthogonal_by_singular_values():
    g = torch.Generator().manual_seed(1)
    for shape in ((7, 12), (12, 7), (9, 9)):
        x = torch.randn(shape, generator=g).double()
        u, s, v = torch.linalg.svd(x, full_matrices=False)
        a, b, c = ref.QUINTIC
        t = s / s.norm()
        for _ in range(5):
            t = a * t + b * t ** 3 + c * t ** 5
        assert (ref.orthogonal(x, 5, 0.0) - u * t @ v).abs().max() < 1e-9
        assert (ref.orthogonal(x, 5, 0.0, held=True) - u * t @ v).norm() < 0.05 * t.norm()


def test_held_forms_stay_inside_binary16():
    """Over the whole range of singular values: X below 2^6 * 1.21, S and its polynomial below 65504."""
    a, b, c = ref.QUINTIC
    s = torch.linspace(0, 1.21, 100_001, dtype=torch.float64)
    assert (a * s + b * s ** 3 + c * s ** 5).abs().max() < 1.21
    assert s.square().max() * ref.HELD[1] < 65504 / 2 and (b * s ** 2 + c * s ** 4).abs().max() * ref.HELD[2] < 65504 / 2


def test_orthogonalize_refusals(L):
    g, out, ws = BASE, BASE + 64 * MB, BASE + 128 * MB
    need = L.ring_orthogonalize_workspace(3, 100, 200)
    assert need > 3 * 2 * 128 * 256 * 2 and L.ring_orthogonalize_workspace(0, 5, 5) == 0
    assert L.ring_orthogonalize_workspace(65536, 5, 5) == 0

    def call(g=g, ldg=200, sg=20000, dt=F32, out=out, ldo=200, so=20000, odt=BF16, batch=3, rows=100, cols=200, steps=5, eps=1e-7,
             ws=ws, wb=need):
        return L.ring_orthogonalize(g, ldg, sg, dt, out, ldo, so, odt, batch, rows, cols, steps, eps, ws, wb, None)

    assert call() == ECUDA and call(out=g, odt=F32) == ECUDA and call(batch=1, sg=0, so=0) == ECUDA
    assert call(batch=0) == OK and call(rows=0) == OK and call(cols=0) == OK
    assert call(dt=3) == EINVAL and call(odt=-1) == EINVAL and call(steps=0) == EINVAL and call(steps=1001) == EINVAL
    assert call(eps=-1e-9) == EINVAL and call(eps=float("nan")) == EINVAL and call(eps=float("inf")) == EINVAL
    assert call(g=None) == EINVAL and call(g=g + 2) == EINVAL and call(out=out + 1) == EINVAL and call(ldg=199) == EINVAL
    assert call(ldo=199) == EINVAL and call(sg=19999) == EINVAL and call(so=19999) == EINVAL and call(batch=65536) == EINVAL
    assert call(rows=1 << 31) == EINVAL and call(wb=need - 1) == EINVAL and call(ws=None) == EINVAL and call(ws=ws + 16) == EINVAL
    assert call(out=g) == EALIAS and call(out=g + 400) == EALIAS and call(ws=g) == EALIAS and call(ws=out) == EALIAS
    assert call(out=g, odt=F32, ldo=201, so=30000) == EALIAS
