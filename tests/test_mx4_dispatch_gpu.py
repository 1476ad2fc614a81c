"""The 4-bit kernels at the sizes that choose each of them: the row kernel that
quantises rows straight from memory where tiles are many.

Sizes on and beyond each edge of the rules follow from the GPU's SM count.
"""
import numpy as np
import pytest
import torch

import mx4_reference as ref

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
