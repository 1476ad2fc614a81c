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
