"""GPU tests of the microscaled 4-bit operators and dropout against their
definitions in 64 bits (mx4_reference).

Quantisation, dequantisation, dropout masks and the 4-bit AllReduce are compared
bit for bit; the product within a bound derived from its sums (see product_bound).
"""
import numpy as np
import pytest
import torch

import mx4_reference as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
# half a unit in the last place, relative
HALF_ULP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import ring_allreduce_reducescatter_gb300 as mod

    torch.cuda.set_device(0)
    return mod


@pytest.fixture(autouse=True)
def device_status_stays_clear(request):
    yield
    if "rr" in request.fixturenames:
        assert request.getfixturevalue("rr").device_status() == 0, "a kernel set the device status word"


def values_of(rows, cols, dtype, seed, sigma=1.0):
    """Normal values with magnitudes over many binades from row to row, exact zeros and whole zero blocks."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * sigma
    x *= torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g).float())
    x[torch.rand((rows, cols), generator=g) < 0.05] = 0
    if rows > 2:
        x[rows // 2] = 0
    if cols > 40:
        x[:, cols // 3:cols // 3 + 33] = 0
    return x.to(dtype)


def as64(x):
    return x.detach().cpu().double().numpy()


def check_stored(q, codes, scales):
    data, tiles = ref.pack(codes, scales)
    got_d, got_s = q.data.cpu().numpy(), q.scales.cpu().numpy()
    assert np.array_equal(got_s, tiles)
    # -0 and +0 codes stand for the same value; the sign is kept, so they are equal too
    assert np.array_equal(got_d, data)


SIZES = [(1, 1), (1, 31), (1, 32), (1, 33), (2, 255), (3, 256), (5, 257), (31, 64), (33, 40), (127, 129), (128, 256),
         (129, 300), (257, 511), (300, 1000)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_bits(rr, rows, cols, dtype, rounding):
    x = values_of(rows, cols, dtype, rows * 1000 + cols)
    d = x.cuda()
    seed, sub = 0x1234_5678_9ABC_DEF0 + rows, (cols << 33) + 7
    rnd = (lambda k: (seed, sub + k)) if rounding == "stochastic" else (lambda k: None)
    how = dict(rounding=rounding, seed=seed, subsequence=sub)
    check_stored(rr.mx4_quantize(d, **how), *ref.quantize(as64(x), rnd(0)))
    check_stored(rr.mx4_quantize(d, transposed=True, **how), *ref.quantize(as64(x).T, rnd(0)))
    by_rows, by_cols = rr.mx4_quantize_both(d, **how)
    check_stored(by_rows, *ref.quantize(as64(x), rnd(0)))
    check_stored(by_cols, *ref.quantize(as64(x).T, rnd(1)))
    assert by_rows.shape == (rows, cols) and by_cols.shape == (cols, rows)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 3), (8, 8), (3, 5), (2, 1), (4, 12), (7, 9)])
def test_quantize_strides_and_alignment(rr, dtype, offset, pad):
    """Rows further apart than their length, starts off the 16-byte grid."""
    rows, cols = 170, 301
    slab = torch.full((offset + rows * (cols + pad) + 16,), float("nan"), dtype=dtype, device="cuda")
    view = slab[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    x = values_of(rows, cols, dtype, 5)
    view.copy_(x)
    by_rows, by_cols = rr.mx4_quantize_both(view)
    check_stored(by_rows, *ref.quantize(as64(x)))
    check_stored(by_cols, *ref.quantize(as64(x).T))
    check_stored(rr.mx4_quantize(view), *ref.quantize(as64(x)))


def test_quantize_extremes(rr):
    """Subnormals, the largest values, the boundary of a scale, infinities and NaN."""
    x = torch.zeros((12, 64))
    x[0, 0] = 2.0 ** -149
    x[1, 0] = 3.4e38
    x[2, 0], x[2, 1] = 1.5, 0.25
    x[3, 0], x[3, 1] = float(np.nextafter(np.float32(1.5), np.float32(2))), 0.25
    x[4, 0], x[4, 40] = float("inf"), 1.0
    x[5, 5], x[5, 40] = float("nan"), 2.0
    x[6, 0], x[6, 1] = -float("inf"), 3.0
    x[7, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)
    x[8, :32] = -x[7, :32]
    x[9, 0], x[9, 1] = 2.0 ** -126 * 6, 2.0 ** -130
    x[10, 3] = -0.0
    x[11, 0], x[11, 1:32] = 6.0, 2.0 ** -20
    for rounding, rnd in (("nearest", None), ("stochastic", (3, 4))):
        q, t = rr.mx4_quantize_both(x.cuda(), rounding=rounding, seed=3, subsequence=4)
        check_stored(q, *ref.quantize(as64(x), rnd))
        check_stored(t, *ref.quantize(as64(x).T, rnd and (3, 5)))
        check_stored(rr.mx4_quantize(x.cuda(), rounding=rounding, seed=3, subsequence=4), *ref.quantize(as64(x), rnd))
    v = rr.mx4_dequantize(q)
    assert torch.isnan(v[4, :32]).all() and v[4, 40] == 1.0 and torch.isnan(v[5, :32]).all() and v[5, 40] == 2.0
    # 3.4e38 rounds to 4 * 2^126, one binade above binary32 (either way with these numbers)
    assert torch.isinf(v[1, 0]) == (float(ref.values(*ref.quantize(as64(x), (3, 4)), 64)[1, 0]) == 2.0 ** 128)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (130, 257), (40, 512), (50, 7), (9, 16), (5, 17), (300, 47), (260, 1001)])
def test_dequantize(rr, rows, cols, dtype):
    data, tiles, v = ref.random_matrix(rows, cols, 7)
    q = rr.Mx4(data.cuda(), tiles.cuda(), rows, cols)
    got = rr.mx4_dequantize(q, dtype)
    assert got.dtype == dtype and np.array_equal(as64(got), v)
    slab = torch.zeros((rows, cols + 5), dtype=dtype, device="cuda")
    rr.mx4_dequantize(q, out=slab[:, 1:cols + 1])
    assert np.array_equal(as64(slab[:, 1:cols + 1]), v) and not slab[:, 0].any() and not slab[:, cols + 1:].any()


def test_stochastic_rounding_is_unbiased(rr):
    """The mean of many roundings of one value: 2^20 draws, within five standard errors."""
    for v in (0.1, 0.3, 1.2, 2.7, 5.1):
        x = torch.full((1024, 1024), v)
        x[:, ::32] = 6.0
        q = rr.mx4_dequantize(rr.mx4_quantize(x.cuda(), rounding="stochastic", seed=11))
        got = as64(q)[:, 1:32].ravel()
        step = 0.5 if v < 2 else 1.0 if v < 4 else 2.0
        # a draw's deviation is at most step / 2; 2^-16 of a step is the numbers' resolution
        assert abs(got.mean() - np.float32(v)) < 5 * step / 2 / np.sqrt(got.size) + step * 2.0 ** -16


# --------------------------------------------------------------------- dropout


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
@pytest.mark.parametrize("n,first", [(1, 0), (7, 0), (8, 0), (1000, 3), (4096, 2 ** 35 + 5), (10_001, 8)])
def test_dropout_flat(rr, dtype, p, n, first):
    x, r = values_of(1, n, dtype, n), values_of(1, n, dtype, n + 1)
    factor, kept = ref.drop_factor(p, 99, 5, first, 1, n)
    d = rr.Dropout(p, 99, 5, first)
    t = torch.from_numpy(factor).float()
    want = torch.where(torch.from_numpy(kept), x.float() * t, torch.zeros(()))
    for residual, w in ((None, want), (r, r.float() + want)):
        got = rr.dropout(x.cuda(), d, residual=None if residual is None else residual.cuda())
        assert torch.equal(got.cpu(), w.to(dtype))


def test_dropout_ranges_and_shards_agree(rr):
    """Any cut of the tensor gives the bits of the whole."""
    x = values_of(1, 5000, BF16, 3).cuda().view(-1)
    whole = rr.dropout(x, rr.Dropout(0.3, 17, 2))
    for cut in (1, 8, 777, 4999):
        a, b = rr.dropout(x[:cut], rr.Dropout(0.3, 17, 2)), rr.dropout(x[cut:], rr.Dropout(0.3, 17, 2, cut))
        assert torch.equal(torch.cat((a, b)), whole)


def test_dropout_strided_in_place_and_shapes(rr):
    rows, cols = 33, 45
    x = values_of(rows, cols + 7, F32, 4).cuda()
    view, d = x[:, 2:cols + 2], rr.Dropout(0.25, 5)
    want = rr.dropout(view.contiguous(), d)
    res = values_of(rows, cols, F32, 6).cuda()
    assert torch.equal(rr.dropout(view, d), want)
    assert torch.equal(rr.dropout(view, d, residual=res), res + want)
    assert torch.equal(rr.dropout(view.contiguous().view(3, 11, cols), d), want.view(3, 11, cols))
    out = torch.empty((rows, cols + 1), device="cuda")[:, :cols]
    assert rr.dropout(view, d, out=out) is out and torch.equal(out, want)
    acc = res.clone()
    rr.dropout(view.contiguous(), d, residual=acc, out=acc)
    assert torch.equal(acc, res + want)
    rr.dropout(view, d, out=view)
    assert torch.equal(view, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,gap", [(33, 45, 0), (300, 136, 0), (70, 129, 3)])
def test_output_beside_its_input(rr, m, n, gap, dtype):
    """dropout and the product's residual from one half of an array's columns into the other."""
    d = rr.Dropout(0.25, 5)
    qa, qb = (rr.mx4_quantize(values_of(r, 96, F32, 8 + r).cuda()) for r in (m, n))
    for left in (True, False):
        whole = values_of(m, 2 * n + gap, dtype, 4).cuda()
        src, dst = (whole[:, :n], whole[:, n + gap:]) if left else (whole[:, n + gap:], whole[:, :n])
        x = src.clone()
        rr.dropout(src, d, out=dst)
        assert torch.equal(dst, rr.dropout(x, d)) and torch.equal(src, x)
        rr.mx4_matmul(qa, qb, residual=src, dropout=d, out=dst)
        assert torch.equal(dst, rr.mx4_matmul(qa, qb, dtype, residual=x, dropout=d)) and torch.equal(src, x)


def test_dropout_ignores_what_it_drops(rr):
    x = torch.full((4096,), float("nan"), device="cuda")
    y = rr.dropout(x, rr.Dropout(0.5, 1))
    kept = torch.from_numpy(ref.drop_factor(0.5, 1, 0, 0, 1, 4096)[1][0])
    assert torch.equal(torch.isnan(y).cpu(), kept) and not y.cpu()[~kept].any()


def test_dropout_gradient_by_differences(rr):
    """dropout is linear: its backward pass is the same map, so <dy, f(x + h) - f(x)> = <f'(dy), h>."""
    d = rr.Dropout(0.2, 8)
    g = torch.Generator().manual_seed(1)
    x, h, dy = (torch.randint(-8, 9, (64, 65), generator=g).float().cuda() for _ in range(3))
    left = (dy.double() * (rr.dropout(x + h, d).double() - rr.dropout(x, d).double())).sum()
    right = (rr.dropout(dy, d).double() * h.double()).sum()
    # every f(x) is one rounding off a whole number times 1.25: relative 2^-24 a term
    assert abs(float(left - right)) <= 2.0 ** -22 * float((dy.abs() * (x.abs() + h.abs())).double().sum()) * 1.25


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("rows,cols,p", [(1, 40, 0.3), (65, 96, 0.3), (130, 333, 0.3), (66, 160, 0.999), (300, 512, 0.1)])
def test_quantize_with_dropout(rr, rows, cols, p, dtype, rounding):
    """Quantisation of a dropped-out matrix: the binary32 product, never rounded
    to storage; at p = 0.999 most blocks and whole rows are empty."""
    x = values_of(rows, cols, dtype, 12)
    factor, kept = ref.drop_factor(p, 21, 4, 9, rows, cols)
    g = np.where(kept, (x.float() * torch.from_numpy(factor).float()).numpy(), 0).astype(np.float64)
    rnd = (lambda k: (1, 2 + k)) if rounding == "stochastic" else (lambda k: None)
    how = dict(rounding=rounding, seed=1, subsequence=2, dropout=rr.Dropout(p, 21, 4, 9))
    q, t = rr.mx4_quantize_both(x.cuda(), **how)
    check_values(q, ref.quantize(g, rnd(0)))
    check_values(t, ref.quantize(g.T, rnd(1)))
    check_values(rr.mx4_quantize(x.cuda(), **how), ref.quantize(g, rnd(0)))
    check_values(rr.mx4_quantize(x.cuda(), transposed=True, **how), ref.quantize(g.T, rnd(0)))


def check_values(q, want):
    """Scales alike and values alike (a dropped element's zero may have either sign)."""
    codes, scales = ref.unpack(q.data.cpu().numpy(), q.scales.cpu().numpy(), q.rows, q.cols)
    assert np.array_equal(scales, want[1])
    assert np.array_equal(ref.values(codes, scales, q.cols), ref.values(*want, q.cols), equal_nan=True)


def test_offsets_past_32_bits(rr):
    """More than 2^32 elements: the last rows are those of the last rows alone."""
    rows, cols, tail = 66_048, 65_544, 128  # 4.33e9 elements; the tail starts a scale tile
    x = torch.empty((rows, cols), dtype=BF16, device="cuda")
    x[:-tail].zero_()
    x[-tail:] = values_of(tail, cols, BF16, 1).cuda()
    last = x[-tail:]
    q = rr.mx4_quantize(x)
    want = rr.mx4_quantize(last)
    assert torch.equal(q.data[-tail:], want.data) and torch.equal(q.scales[-1], want.scales[0])
    assert not q.data[:-tail].any()
    out = rr.mx4_dequantize(q, BF16)
    assert torch.equal(out[-tail:], rr.mx4_dequantize(want, BF16)) and not out[:-tail].any()
    t = rr.mx4_quantize(x, transposed=True)
    assert torch.equal(t.data[:, -tail // 2:], rr.mx4_quantize(last, transposed=True).data)
    del t
    y = rr.mx4_allreduce([q, q], [out, torch.empty_like(out)])[1]  # twice the values, exact
    assert torch.equal(y[-tail:], 2 * rr.mx4_dequantize(want, BF16)) and not y[:-tail].any()
    d = rr.Dropout(0.4, 3, 1)
    rr.dropout(x, d, out=y)
    whole = rr.dropout(last.reshape(-1), d._replace(first=(rows - tail) * cols)).view(tail, cols)
    assert torch.equal(y[-tail:], whole)
    del y, x
    a, b = values_of(rows, 64, F32, 2).cuda(), values_of(cols, 64, F32, 3).cuda()
    qa, qb = rr.mx4_quantize(a), rr.mx4_quantize(b)
    rr.mx4_matmul(qa, qb, out=out, dropout=d)
    small = rr.mx4_matmul(rr.mx4_quantize(a[-tail:].contiguous()), qb, dropout=d._replace(first=(rows - tail) * cols))
    assert torch.equal(out[-tail:], small)


# --------------------------------------------------------------------- product


def product_bound(a, b, y, dtype):
    """What a correct product may be off: binary32 accumulation of ceil(K / 64)
    partial sums, each within 2^-22 of the sum of magnitudes (one binary32
    operation and the alignment inside it), four more for the sum inside 64
    elements, and the rounding to storage (to binary16's subnormals too)."""
    mags = np.abs(a) @ np.abs(b).T
    acc = 2.0 ** -22 * (-(-a.shape[1] // 64) + 4) * mags
    return acc + HALF_ULP[dtype] * (np.abs(y) + acc) + (2.0 ** -25 if dtype == F16 else 0)


PRODUCTS = [(1, 1, 1), (1, 8, 32), (1, 300, 64), (2, 129, 65), (7, 16, 4096), (16, 128, 256), (17, 127, 257),
            (33, 512, 1000), (64, 130, 2000), (127, 64, 511), (128, 128, 128), (129, 200, 768), (200, 333, 1537),
            (256, 256, 512), (300, 520, 300), (513, 257, 1030),
            (2561, 2050, 300), (1111, 5000, 1030), (130, 19_500, 65), (1000, 1021, 4100), (300, 2500, 4096)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(rr, m, n, k, dtype):
    da, sa, a = ref.random_matrix(m, k, m + k, spread=2)
    db, sb, b = ref.random_matrix(n, k, n + 3 * k, spread=2)
    qa, qb = rr.Mx4(da.cuda(), sa.cuda(), m, k), rr.Mx4(db.cuda(), sb.cuda(), n, k)
    y = a @ b.T
    out = rr.mx4_matmul(qa, qb, dtype)
    assert out.dtype == dtype and out.shape == (m, n)
    bad = np.abs(as64(out) - y) > product_bound(a, b, y, dtype)
    assert not bad.any(), f"{bad.sum()} of {bad.size} elements, first {np.argwhere(bad)[:5].tolist()}"
    assert torch.equal(out, rr.mx4_matmul(qa, qb, dtype)), "two calls differ"


@pytest.mark.parametrize("m,n,k", [(3, 40, 64), (130, 260, 300), (300, 1000, 512), (2500, 2300, 1600)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_places_every_element(rr, m, n, k, dtype):
    """Sums of one term each: out[i, j] is exact, so any mix-up of rows, columns, K or scales shows."""
    g = np.random.default_rng(k)
    codes_a = g.integers(0, 16, (m, -(-k // 32) * 32))
    codes_a[:, k:] = 0
    scales_a = 127 + g.integers(-3, 4, (m, -(-k // 32)))
    at = g.integers(0, k, n)
    codes_b, scales_b = np.zeros((n, -(-k // 32) * 32), dtype=np.int64), 127 + g.integers(-3, 4, (n, -(-k // 32)))
    codes_b[np.arange(n), at] = 2  # 1.0
    stored = [tuple(torch.from_numpy(t).cuda() for t in ref.pack(c, s)) for c, s in ((codes_a, scales_a), (codes_b, scales_b))]
    y = ref.values(codes_a, scales_a, k) @ ref.values(codes_b, scales_b, k).T
    out = rr.mx4_matmul(rr.Mx4(*stored[0], m, k), rr.Mx4(*stored[1], n, k), dtype)
    assert np.array_equal(as64(out), y)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k,p", [(1, 40, 64, 0.0), (5, 33, 96, 0.2), (130, 129, 256, 0.1), (300, 264, 512, 0.5),
                                     (2600, 2050, 320, 0.1), (2304, 2560, 64, 0.3), (40, 90, 128, 0.999)])
def test_product_epilogue(rr, m, n, k, p, dtype):
    """residual + dropout(product): the elements of the plain product in binary32, masked and added."""
    da, sa, _ = ref.random_matrix(m, k, 1, spread=1)
    db, sb, _ = ref.random_matrix(n, k, 2, spread=1)
    qa, qb = rr.Mx4(da.cuda(), sa.cuda(), m, k), rr.Mx4(db.cuda(), sb.cuda(), n, k)
    r = values_of(m, n, dtype, 3).cuda()
    factor, kept = ref.drop_factor(p, 77, 1, 11, m, n)
    acc = rr.mx4_matmul(qa, qb, F32)
    dropped = torch.where(torch.from_numpy(kept).cuda(), acc * torch.from_numpy(factor).float().cuda(), torch.zeros((), device="cuda"))
    d = rr.Dropout(p, 77, 1, 11)
    assert torch.equal(rr.mx4_matmul(qa, qb, dtype, dropout=d), dropped.to(dtype))
    assert torch.equal(rr.mx4_matmul(qa, qb, dtype, residual=r), (r.float() + acc).to(dtype))
    want = (r.float() + dropped).to(dtype)
    assert torch.equal(rr.mx4_matmul(qa, qb, dtype, residual=r, dropout=d), want)
    # strided, unaligned output and residual; then in place
    slab = torch.zeros((m, n + 9), dtype=dtype, device="cuda")
    wide = torch.zeros((m, n + 3), dtype=dtype, device="cuda")
    wide[:, 1:n + 1] = r
    rr.mx4_matmul(qa, qb, residual=wide[:, 1:n + 1], dropout=d, out=slab[:, 4:n + 4])
    assert torch.equal(slab[:, 4:n + 4], want) and not slab[:, :4].any() and not slab[:, n + 4:].any()
    rr.mx4_matmul(qa, qb, residual=r, dropout=d, out=r)
    assert torch.equal(r, want)


def test_product_of_nothing(rr):
    """K = 0: the sum is 0; no rows or columns: nothing happens."""
    e = lambda rows, cols: rr.Mx4.empty(rows, cols, torch.device("cuda"))
    r = values_of(5, 7, F32, 1).cuda()
    assert not rr.mx4_matmul(e(5, 0), e(7, 0), F32).any()
    assert torch.equal(rr.mx4_matmul(e(5, 0), e(7, 0), F32, residual=r), r)
    assert rr.mx4_matmul(e(0, 64), e(7, 64)).shape == (0, 7)
    q, t = rr.mx4_quantize_both(torch.empty((0, 5), device="cuda"))
    assert q.shape == (0, 5) and t.shape == (5, 0) and rr.mx4_dequantize(q).shape == (0, 5)
    assert rr.dropout(torch.empty(0, device="cuda"), rr.Dropout(0.5, 1)).numel() == 0
    assert [t.shape for t in rr.mx4_allreduce([e(0, 4), e(0, 4)])] == [(0, 4)] * 2


@pytest.mark.parametrize("m,n", [(1, 200), (40, 200), (200, 300)])
def test_product_carries_nan_blocks(rr, m, n):
    """A block that was not finite makes its row (or column) NaN and no other."""
    k = 320
    x, w = values_of(m, k, F32, 1), values_of(n, k, F32, 2)
    x[0, 100], w[5, 3] = float("inf"), float("nan")
    y = rr.mx4_matmul(rr.mx4_quantize(x.cuda()), rr.mx4_quantize(w.cuda()), F32)
    want = torch.zeros((m, n), dtype=torch.bool)
    want[0], want[:, 5] = True, True
    assert torch.equal(torch.isnan(y).cpu(), want)


# ------------------------------------------------------------- 4-bit AllReduce


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("R,rows,cols", [(1, 3, 5), (2, 1, 1), (3, 7, 33), (4, 64, 64), (5, 1, 3), (8, 130, 257), (64, 9, 40),
                                         (3, 50, 7), (5, 33, 17), (7, 40, 48), (4, 100, 31), (64, 3, 5), (2, 300, 1000)])
def test_allreduce_is_the_ring_of_the_values(rr, R, rows, cols, dtype):
    """Bit for bit the ring AllReduce of the values, binary32 wire."""
    qs, vals = [], []
    for r in range(R):
        data, tiles, v = ref.random_matrix(rows, cols, r, spread=9)
        qs.append(rr.Mx4(data.cuda(), tiles.cuda(), rows, cols))
        vals.append(torch.from_numpy(v).float().cuda().view(-1))
    want = rr.allreduce(vals)
    outs = rr.mx4_allreduce(qs, dtype=dtype)
    assert len(outs) == R
    for o, w in zip(outs, want):
        assert torch.equal(o.view(-1), w.to(dtype))
    off = [torch.zeros(rows * cols + 1, dtype=dtype, device="cuda")[1:].view(rows, cols) for _ in range(R)]
    rr.mx4_allreduce(qs, off)
    for o, w in zip(off, want):
        assert torch.equal(o.view(-1), w.to(dtype))


# ------------------------------------------------------------------- the layer


def test_linear_gradients_match_the_formula(rr):
    """mx4_linear against the layer's formulas in 64 bits on the quantised operands."""
    m, n, k, p = 100, 136, 200, 0.25
    x, w, r, dy = (values_of(a, b, BF16, s).float().clamp(-8, 8).to(BF16) for s, (a, b) in enumerate(((m, k), (n, k), (m, n), (m, n))))
    xs, ws, rs = (t.cuda().requires_grad_() for t in (x, w, r))
    y = rr.mx4_linear(xs, ws, residual=rs, drop=rr.Dropout(p, 5, 6), seed=7, subsequence=20)
    y.backward(dy.cuda())
    val = lambda t, rnd=None: ref.values(*ref.quantize(t, rnd), t.shape[1])
    factor, kept = ref.drop_factor(p, 5, 6, 0, m, n)
    g = np.where(kept, (dy.float() * torch.from_numpy(factor).float()).numpy(), 0).astype(np.float64)
    qx, qw, qxt, qwt = val(as64(x)), val(as64(w)), val(as64(x).T), val(as64(w).T)
    gr, gc = val(g, (7, 20)), val(g.T, (7, 21))
    for got, want, bound in ((y, as64(r) + (qx @ qw.T) * factor, product_bound(qx, qw, as64(r) + (qx @ qw.T) * factor, BF16) * 2),
                             (xs.grad, gr @ qwt.T, product_bound(gr, qwt, gr @ qwt.T, BF16)),
                             (ws.grad, gc @ qxt.T, product_bound(gc, qxt, gc @ qxt.T, BF16))):
        assert (np.abs(as64(got) - want) <= bound).all()
    assert torch.equal(rs.grad.cpu(), dy)


def test_linear_gradients_one_at_a_time(rr):
    """Either gradient alone, and neither, give the bits of both together."""
    x, w, dy = values_of(70, 96, BF16, 1).cuda(), values_of(130, 96, BF16, 2).cuda(), values_of(70, 130, BF16, 3).cuda()
    d = rr.Dropout(0.2, 9, 1)

    def run(need_x, need_w):
        xs, ws = x.clone().requires_grad_(need_x), w.clone().requires_grad_(need_w)
        y = rr.mx4_linear(xs, ws, drop=d, seed=4, subsequence=10)
        if need_x or need_w:
            y.backward(dy)
        return y.detach(), xs.grad, ws.grad

    y, dx, dw = run(True, True)
    assert torch.equal(run(True, False)[1], dx) and torch.equal(run(False, True)[2], dw)
    assert torch.equal(run(False, False)[0], y) and run(True, False)[2] is None
    with torch.no_grad():
        assert torch.equal(rr.mx4_linear(x.clone().requires_grad_(), w, drop=d, seed=4, subsequence=10), y)
    # a gradient that is one value spread over the matrix (stride zero)
    xs = x.clone().requires_grad_()
    rr.mx4_linear(xs, w, drop=d).sum().backward()
    ones = x.clone().requires_grad_()
    rr.mx4_linear(ones, w, drop=d).backward(torch.ones_like(y))
    assert torch.equal(xs.grad, ones.grad)


def test_linear_gradient_by_differences(rr):
    """Where every operand is a 4-bit value and every block's scale is held by a 6,
    the layer is exactly bilinear: differences along x and w equal the gradients."""
    m, n, k = 32, 64, 96
    g = torch.Generator().manual_seed(3)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4])

    def draw(rows, cols):
        t = grid[torch.randint(0, 7, (rows, cols), generator=g)] * (1 - 2 * torch.randint(0, 2, (rows, cols), generator=g))
        t[torch.arange(rows)[:, None] % 32 == torch.arange(cols)[None, :] % 32] = 6.0
        return t.cuda()

    x, w, dy = draw(m, k), draw(n, k), draw(m, n)
    x.requires_grad_(), w.requires_grad_()
    loss = lambda a, b: (rr.mx4_linear(a, b).double() * dy.double()).sum()
    loss(x, w).backward()
    for t, at in ((x, (3, 40)), (x, (31, 0)), (w, (60, 5)), (w, (2, 95))):
        h = torch.zeros_like(t)
        h[at] = -float(t.detach()[at]) if float(t.detach()[at]) else 1.0  # to another 4-bit value; no block loses its 6
        if abs(float(t.detach()[at])) == 6.0:
            h[at] = -12.0 if float(t.detach()[at]) > 0 else 12.0
        with torch.no_grad():
            diff = loss(x + h, w) - loss(x, w) if t is x else loss(x, w + h) - loss(x, w)
        assert float(diff) == float(t.grad[at].double() * h[at].double()), at


# -------------------------------------------------------------- streams, order


def test_another_stream(rr):
    """Operators on a side stream, their outputs allocated for it."""
    side = torch.cuda.Stream()
    x = values_of(300, 500, BF16, 1).cuda()
    w = values_of(200, 500, BF16, 2).cuda()
    want = rr.mx4_matmul(rr.mx4_quantize(x), rr.mx4_quantize(w))
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        y = rr.mx4_matmul(rr.mx4_quantize(x, stream=side), rr.mx4_quantize(w, stream=side), stream=side)
        d = rr.dropout(y, rr.Dropout(0.5, 1), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want) and torch.equal(d, rr.dropout(want, rr.Dropout(0.5, 1)))


def test_graph_capture(rr):
    """A captured step replays on new inputs."""
    x, w = values_of(64, 256, BF16, 1).cuda(), values_of(96, 256, BF16, 2).cuda()
    qw = rr.mx4_quantize(w)
    step = lambda: rr.dropout(rr.mx4_matmul(rr.mx4_quantize(x), qw), rr.Dropout(0.1, 3))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    x.copy_(values_of(64, 256, BF16, 9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, step())


# -------------------------------------------------------------------- refusals


def test_refusals(rr):
    x = torch.zeros((4, 64), device="cuda")
    q = rr.mx4_quantize(x)
    with pytest.raises(ValueError):
        rr.mx4_quantize(x.double())
    with pytest.raises(ValueError):
        rr.mx4_quantize(x.cpu())
    with pytest.raises(ValueError):
        rr.mx4_quantize(x.t())
    with pytest.raises(ValueError):
        rr.mx4_quantize(x.view(-1))
    with pytest.raises(ValueError):
        rr.mx4_quantize(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        rr.mx4_quantize(x, rounding="up")
    with pytest.raises(rr.RingError):
        rr.mx4_quantize(x, out=rr.Mx4.empty(4, 65))
    with pytest.raises(rr.RingError):
        rr.mx4_quantize(x, dropout=rr.Dropout(1.0, 0))
    with pytest.raises(ValueError):
        rr.Mx4(q.data, q.scales, 4, 65)
    with pytest.raises(ValueError):
        rr.Mx4(q.data.view(torch.int8), q.scales, 4, 64)
    with pytest.raises(ValueError):
        rr.mx4_matmul(q, rr.Mx4.empty(4, 32))
    with pytest.raises(ValueError):
        rr.mx4_matmul(q, q, torch.float64)
    with pytest.raises(ValueError):
        rr.mx4_matmul(q, q, residual=torch.zeros((4, 4), device="cuda"))  # float32 beside bfloat16
    with pytest.raises(ValueError):
        rr.mx4_matmul(q, q, out=torch.zeros((4, 5), device="cuda"))
    with pytest.raises(ValueError):
        rr.dropout(x, rr.Dropout(0.1, 0), residual=x[:2])
    for p in (-0.1, 1.0, 0.999999, float("nan")):
        with pytest.raises(rr.RingError):
            rr.dropout(x, rr.Dropout(p, 0))
    with pytest.raises(rr.RingError):
        flat = x.view(-1)
        rr.dropout(flat[:100], rr.Dropout(0.1, 0), out=flat[4:104])
    with pytest.raises(ValueError):
        rr.mx4_allreduce([])
    with pytest.raises(ValueError):
        rr.mx4_allreduce([q, rr.Mx4.empty(4, 32)])
    out = torch.empty((4, 64), device="cuda")
    with pytest.raises(rr.RingError):
        rr.mx4_allreduce([q, q], [out, out])


def test_data_parallel_example(rr):
    """The example's layer learns on the 4-bit wire, close to the binary32 wire."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx4_data_parallel.py")
    spec = importlib.util.spec_from_file_location("mx4_data_parallel", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    plain = example.train(3, 256, 256, 12, False)
    small = example.train(3, 256, 256, 12, True)
    assert plain[0] == small[0]  # the first step's forward pass is the same
    # the loss falls to well under half, and the 4-bit wire ends within a tenth of where it began
    assert plain[-1] < plain[0] / 2 and small[-1] < small[0] / 2
    assert abs(small[-1] - plain[-1]) < plain[0] / 10
