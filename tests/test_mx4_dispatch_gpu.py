"""The 4-bit kernels at the sizes that choose each of them: the row kernel that
quantises rows straight from memory where tiles are many, and products of more
than 64 rows whose K is split over clusters of two to eight CTAs.

Sizes on and beyond each edge of the rules follow from the GPU's SM count.
"""
import numpy as np
import pytest
import torch

import mx4_reference as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
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


# --------------------------------------------------------------- quantisation

# (storage, rounding, dropout, edges): through tiles up to the first edge (tiles
# of 16 rows by 512 bytes an SM), straight from memory beyond it and up to the
# second one
ROW_FORMS = [
    (F32, "nearest", 0.0, (8, None)), (F32, "stochastic", 0.0, (96, None)), (F32, "nearest", 0.2, (96, None)),
    (F32, "stochastic", 0.2, (96, None)), (F16, "nearest", 0.0, (48, None)), (BF16, "nearest", 0.0, (48, None)),
    (F16, "nearest", 0.2, (6, 8)), (BF16, "nearest", 0.2, (6, 8)), (F16, "stochastic", 0.2, (6, 8)),
    (BF16, "stochastic", 0.2, (6, 8)),
]


def scale_tiles(edge, dtype):
    """The most scale tiles (128 rows by 256 columns) that are at most `edge` tiles an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return edge * sms // (16 if dtype == F32 else 8)


def wide_array(rows, cols, pad, dtype, seed):
    """rows x cols with neighbouring columns in rows of cols + pad, NaN beside them: magnitudes over many binades
    from row to row, zeros and whole zero blocks."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    whole = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g, device="cuda").float())
    x[:, ::17] = 0
    x[::5, cols // 3:cols // 3 + 40] = 0
    whole[:, :cols] = x.to(dtype)
    return whole[:, :cols]


def check_rows(rr, monkeypatch, x, rounding, p):
    """Rows alone against the reference on three tiles of rows, and whole against the rows of both ways at once
    (another kernel, which other tests hold to the reference)."""
    rows, cols = x.shape
    how = dict(rounding=rounding, seed=0x1357_9BDF_0246_8ACE, subsequence=(5 << 40) + 3)
    if p:
        how["dropout"] = rr.Dropout(p, 21, 4, 9)
    q = rr.mx4_quantize(x, **how)
    both = rr.mx4_quantize_both(x, **how)[0]
    assert torch.equal(q.data, both.data) and torch.equal(q.scales, both.scales)
    del both
    tiles, nb, plain = -(-rows // 128), -(-cols // 32), ref.numbers
    for t in sorted({0, tiles // 2, tiles - 1}):
        r0, r1 = t * 128, min(rows, t * 128 + 128)
        v = x[r0:r1].float().cpu().numpy()
        if p:
            factor, kept = ref.drop_factor(p, 21, 4, 9 + r0 * cols, r1 - r0, cols)
            v = np.where(kept, v * factor.astype(np.float32), np.float32(0))
        # the numbers of these rows, from element r0 * 32 * nb of the whole matrix on
        monkeypatch.setattr(ref, "numbers", lambda s, u, first, n: plain(s, u, first + r0 * 32 * nb, n))
        codes, scales = ref.quantize(v, (how["seed"], how["subsequence"]) if rounding == "stochastic" else None)
        monkeypatch.setattr(ref, "numbers", plain)
        data, packed = ref.pack(codes, scales)
        assert np.array_equal(q.scales[t].cpu().numpy(), packed[0])
        assert np.array_equal(q.data[r0:r1].cpu().numpy(), data)


@pytest.mark.parametrize("dtype,rounding,p,edges", ROW_FORMS)
@pytest.mark.parametrize("aligned", [16, 32])
@pytest.mark.parametrize("side", ["on", "beyond"])
def test_rows_at_the_edges(rr, monkeypatch, dtype, rounding, p, edges, aligned, side):
    """One tile of columns: exactly as many scale tiles as an edge allows, and one more."""
    E = 4 if dtype == F32 else 2
    cols = 240 if aligned == 32 else 256 - 16 // E  # rows of whole 32 bytes, or of 16 bytes more
    for k, edge in enumerate(edges):
        if edge is not None:
            n = scale_tiles(edge, dtype) + (side == "beyond")
            check_rows(rr, monkeypatch, wide_array(128 * n - 5, cols, 0, dtype, 10 * k + aligned), rounding, p)


@pytest.mark.parametrize("dtype,rounding,p,edges", ROW_FORMS)
def test_rows_of_a_wide_matrix(rr, monkeypatch, dtype, rounding, p, edges):
    """Nine tiles of columns, the last one short, in the rows of a wider array."""
    cols, across = 8 * 256 + 104, 9  # whole 16-byte groups; not whole halves of a block
    most = scale_tiles(edges[1], dtype) if edges[1] else 2 * scale_tiles(edges[0], dtype)
    down = most // across
    assert down * across > scale_tiles(edges[0], dtype)
    E = 4 if dtype == F32 else 2
    for pad in ((-cols * E) % 32 // E, (-cols * E) % 32 // E + 16 // E):  # rows 32 and only 16 bytes aligned
        check_rows(rr, monkeypatch, wide_array(128 * down - 77, cols, pad, dtype, pad), rounding, p)


def test_rows_of_many_tiles_in_fewer_warps(rr, monkeypatch):
    """Two scale tiles an SM and more: eight warps a tile instead of sixteen."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    check_rows(rr, monkeypatch, wide_array(128 * 2 * sms + 1, 252, 4, F32, 1), "nearest", 0.0)


# -------------------------------------------------------------------- product

# more than 64 rows and fewer than sixteen pairs' tiles: K in 2, 3, 4, 5, 6, 7
# and 8 parts (four steps of 256 or more each)
SPLITS = [(70, 200, 2048), (129, 333, 3100), (128, 264, 4000), (200, 130, 5200), (72, 136, 6200), (100, 264, 7200),
          (512, 512, 8192), (513, 520, 8100)]


def product_bound(a, b, y, dtype):
    """Binary32 accumulation of ceil(K / 64) partial sums, each within 2^-22 of the sum of magnitudes, four more for
    the sum inside 64 elements, one addition a part for at most eight parts (2^-24 each, below one more of those),
    and the rounding to storage (to binary16's subnormals too)."""
    mags = np.abs(a) @ np.abs(b).T
    acc = 2.0 ** -22 * (-(-a.shape[1] // 64) + 5) * mags
    return acc + HALF_ULP[dtype] * (np.abs(y) + acc) + (2.0 ** -25 if dtype == F16 else 0)


def operands(rr, m, n, k, spread):
    (da, sa, a), (db, sb, b) = ref.random_matrix(m, k, m + k, spread), ref.random_matrix(n, k, n + 3 * k, spread)
    return rr.Mx4(da.cuda(), sa.cuda(), m, k), rr.Mx4(db.cuda(), sb.cuda(), n, k), a, b


@pytest.mark.parametrize("m,n,k", SPLITS)
def test_split_product(rr, m, n, k):
    """The product, and residual + dropout(product) out of and in place, at each alignment of the rows."""
    qa, qb, a, b = operands(rr, m, n, k, 2)
    y = a @ b.T
    acc = rr.mx4_matmul(qa, qb, F32)
    factor, kept = ref.drop_factor(0.3, 77, 1, 11, m, n)
    kept, factor = torch.from_numpy(kept).cuda(), torch.from_numpy(factor).float().cuda()
    dropped = torch.where(kept, acc * factor, torch.zeros((), device="cuda"))
    d = rr.Dropout(0.3, 77, 1, 11)
    g = torch.Generator(device="cuda").manual_seed(m)
    for dtype in (F32, F16, BF16):
        out = rr.mx4_matmul(qa, qb, dtype)
        bad = np.abs(out.double().cpu().numpy() - y) > product_bound(a, b, y, dtype)
        assert not bad.any(), f"{dtype}: {bad.sum()} of {bad.size} elements, first {np.argwhere(bad)[:5].tolist()}"
        assert torch.equal(out, acc.to(dtype)) and torch.equal(out, rr.mx4_matmul(qa, qb, dtype)), "two calls differ"
        r = (torch.randn((m, n), generator=g, device="cuda") * 64).to(dtype)
        want = (r.float() + dropped).to(dtype)
        group = 16 // r.element_size()
        ld = -(-n // (4 * group)) * 4 * group
        for at, width in ((0, ld), (0, ld + group), (group, ld + 2 * group), (1, n + 3)):  # 32, 16, 16 bytes, none
            slab = torch.zeros((m, width), dtype=dtype, device="cuda")
            view = slab[:, at:at + n]
            rr.mx4_matmul(qa, qb, residual=r, dropout=d, out=view)
            assert torch.equal(view, want) and not slab[:, :at].any() and not slab[:, at + n:].any()
            view.copy_(r)
            rr.mx4_matmul(qa, qb, residual=view, dropout=d, out=view)
            assert torch.equal(view, want) and not slab[:, :at].any() and not slab[:, at + n:].any()


@pytest.mark.parametrize("m,n,k", SPLITS)
def test_split_product_places_every_element(rr, m, n, k):
    """Sums of one term each: out[i, j] is exact, so a mix-up of rows, columns, parts of K or scales shows."""
    g = np.random.default_rng(k)
    nb = -(-k // 32)
    codes_a = g.integers(0, 16, (m, nb * 32))
    codes_a[:, k:] = 0
    scales_a, scales_b = 127 + g.integers(-3, 4, (m, nb)), 127 + g.integers(-3, 4, (n, nb))
    codes_b = np.zeros((n, nb * 32), dtype=np.int64)
    codes_b[np.arange(n), g.integers(0, k, n)] = 2  # 1.0
    qa, qb = (rr.Mx4(*(torch.from_numpy(t).cuda() for t in ref.pack(c, s)), c.shape[0], k)
              for c, s in ((codes_a, scales_a), (codes_b, scales_b)))
    y = ref.values(codes_a, scales_a, k) @ ref.values(codes_b, scales_b, k).T
    assert np.array_equal(rr.mx4_matmul(qa, qb, F32).double().cpu().numpy(), y)


def test_products_after_one_another(rr):
    """Pairs, splits and whole tiles in turn, each CTA taking over the shared memory of one before it: every
    product has the bits it has alone."""
    sizes = [(2048, 2304, 1100), (1, 4096, 2048), (300, 2500, 4096), (70, 200, 2048), (512, 512, 8192), (33, 1000, 700)]
    ops, want = [], []
    for i, (m, n, k) in enumerate(sizes):
        g = torch.Generator(device="cuda").manual_seed(i)
        a, b = (rr.mx4_quantize(torch.randn((r, k), generator=g, device="cuda")) for r in (m, n))
        ops.append((a, b))
        want.append(rr.mx4_matmul(a, b, BF16))
        torch.cuda.synchronize()
    for rounds in range(20):
        got = [[rr.mx4_matmul(a, b, BF16) for a, b in ops] for _ in range(5)]
        for outs in got:
            for o, w in zip(outs, want):
                assert torch.equal(o, w)
