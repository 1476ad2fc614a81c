"""dropout and the product's residual where the output is an input: in every
storage format, on the vector paths and off them, the bits of the same call out
of place."""
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


def draw(rows, cols, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((rows, cols), generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols,pad,at", [(1, 1, 0, 0), (1, 300_003, 0, 0), (64, 4096, 0, 0), (33, 4104, 8, 0),
                                              (65, 4088, 16, 8), (200, 999, 0, 0), (70, 1001, 4, 3)])
def test_dropout_in_place(rr, rows, cols, pad, at, dtype):
    """Contiguous (one long row), strided on the 16-byte grid and off it; x, the residual or both as the output."""
    d = rr.Dropout(0.3, 6, 1, 2)
    x, r = draw(rows, cols, 1, dtype), draw(rows, cols, 2, dtype)
    plain, with_r, twice = rr.dropout(x, d), rr.dropout(x, d, residual=r), rr.dropout(x, d, residual=x)

    def held(t):
        whole = torch.full((rows, cols + pad + at), 7.0, dtype=dtype, device="cuda")
        whole[:, at:at + cols] = t
        return whole, whole[:, at:at + cols]

    for start, args, want in ((x, lambda v: dict(x=v), plain), (x, lambda v: dict(x=v, residual=r), with_r),
                              (r, lambda v: dict(x=x, residual=v), with_r), (x, lambda v: dict(x=v, residual=v), twice)):
        whole, v = held(start)
        rr.dropout(drop=d, out=v, **args(v))
        assert torch.equal(v, want)
        assert (whole[:, :at] == 7).all() and (whole[:, at + cols:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(5, 304, 512), (40, 304, 512), (200, 304, 512), (2600, 2064, 320)])
@pytest.mark.parametrize("at", [0, 16, 4])
def test_residual_in_place(rr, m, n, k, at, dtype):
    """Rows of whole 32-byte, of 16-byte groups, and off the grid: the small products, the tiles and the pairs."""
    a, b = rr.mx4_quantize(draw(m, k, 1, F32)), rr.mx4_quantize(draw(n, k, 2, F32))
    r, d = draw(m, n, 3, dtype), rr.Dropout(0.2, 5)
    want = rr.mx4_matmul(a, b, dtype, residual=r, dropout=d)
    E = r.element_size()
    whole = torch.full((m, -(-(n + at // E) * E // 32) * 32 // E), 7.0, dtype=dtype, device="cuda")
    v = whole[:, at // E:at // E + n]
    v.copy_(r)
    rr.mx4_matmul(a, b, residual=v, dropout=d, out=v)
    assert torch.equal(v, want)
    assert (whole[:, :at // E] == 7).all() and (whole[:, at // E + n:] == 7).all()
