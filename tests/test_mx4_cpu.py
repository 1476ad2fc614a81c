"""CPU tests of the microscaled 4-bit operators: the reference against published
and hand-worked values, and the C ABI's refusals (no kernel is launched)."""
import ctypes

import numpy as np
import pytest

import mx4_reference as ref

OK, EINVAL, EUNSUP, EALIAS, ECUDA = range(5)
F32, F16, BF16 = 0, 1, 2
BASE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from ring_allreduce_reducescatter_gb300 import _build

    _build.build()
    import ring_allreduce_reducescatter_gb300 as rr

    return rr.lib()


def matrix(data, scales, rows, cols):
    from ring_allreduce_reducescatter_gb300 import mx4

    return mx4._Matrix(data, scales, rows, cols)


def drop(p, seed=1):
    from ring_allreduce_reducescatter_gb300 import mx4

    return ctypes.byref(mx4._Drop(p, seed, 0, 0))


def test_generator_known_answers():
    """The published known answers of Philox4x32-10 (counter and key all zeros,
    all ones, and the digits of pi)."""
    assert ref.philox(0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = (1 << 64) - 1
    assert ref.philox(ones, ones, ones) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox(0x299F31D0A4093822, 0x0370734413198A2E, 0x85A308D3243F6A88) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_numbers_follow_the_generator():
    words = ref.philox(5, 9, 3) + ref.philox(5, 9, 4)
    want = [h for w in words for h in (w & 0xFFFF, w >> 16)]
    assert ref.numbers(5, 9, 24, 16).tolist() == want
    assert ref.numbers(5, 9, 27, 9).tolist() == want[3:12]


def test_reference_quantises_by_hand():
    x = np.zeros((1, 64))
    x[0, :8] = [6.0, -5.0, 2.5, 0.25, 0.75, -0.2, 3.5, 1.25]  # scale 1; ties to the even place
    x[0, 32:35] = [6.5, 0.5, 1.0]  # above 6: scale 2
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127, 128]]
    assert ref.values(codes, scales, 64)[0, :8].tolist() == [6, -4, 2, 0, 1, 0, 4, 1]
    assert ref.values(codes, scales, 64)[0, 32:35].tolist() == [6, 0, 1]


def test_storage_round_trip():
    data, tiles, v = ref.random_matrix(131, 300, 3)
    codes, scales = ref.unpack(data.numpy(), tiles.numpy(), 131, 300)
    assert np.array_equal(ref.values(codes, scales, 300), v)


def test_sizes(L):
    for rows in (0, 1, 127, 128, 129, 5000):
        for cols in (0, 1, 31, 32, 33, 255, 256, 257, 11008):
            data, tiles, _ = (None, None, None) if rows * cols == 0 else ref.random_matrix(min(rows, 129), cols, 1)
            assert L.ring_mx4_row_bytes(cols) == -(-cols // 32) * 16
            assert L.ring_mx4_scale_bytes(rows, cols) == -(-rows // 128) * -(-cols // 256) * 1024
            if data is not None and rows <= 129:
                assert data.numel() == rows * L.ring_mx4_row_bytes(cols)
                assert tiles.numel() == L.ring_mx4_scale_bytes(rows, cols)


def quantize(L, x=BASE, rows=64, cols=96, ld=96, dtype=F32, by_rows="ok", by_cols=None, rounding=0, d=None):
    r = matrix(BASE + (1 << 20), BASE + (2 << 20), 64, 96) if by_rows == "ok" else by_rows
    return L.ring_mx4_quantize(x, rows, cols, ld, dtype, ctypes.byref(r) if r is not None else None,
                               ctypes.byref(by_cols) if by_cols is not None else None, rounding, 0, 0, d, None)


def test_quantize_refusals(L):
    assert quantize(L) == ECUDA  # valid: fails only for want of a GPU
    assert quantize(L, by_rows=None) == EINVAL
    assert quantize(L, dtype=3) == EINVAL and quantize(L, rounding=2) == EINVAL
    assert quantize(L, x=None) == EINVAL and quantize(L, x=BASE + 2) == EINVAL
    assert quantize(L, ld=95) == EINVAL
    assert quantize(L, rows=63) == EINVAL and quantize(L, cols=95) == EINVAL
    assert quantize(L, by_cols=matrix(BASE + (3 << 20), BASE + (4 << 20), 64, 96)) == EINVAL  # not transposed
    assert quantize(L, by_rows=matrix(BASE + 8 + (1 << 20), BASE + (2 << 20), 64, 96)) == EINVAL
    assert quantize(L, by_rows=matrix(BASE + (1 << 20), 0, 64, 96)) == EINVAL
    assert quantize(L, by_rows=matrix(BASE + 64, BASE + (2 << 20), 64, 96)) == EALIAS
    assert quantize(L, by_cols=matrix(BASE + (1 << 20), BASE + (4 << 20), 96, 64)) == EALIAS
    assert quantize(L, by_rows=matrix(BASE + (1 << 20), BASE + (1 << 20) + 16, 64, 96)) == EALIAS
    for p in (-0.5, 1.0, 0.999999, float("nan")):
        assert quantize(L, d=drop(p)) == EINVAL
    big = 1 << 31
    assert quantize(L, rows=big, by_rows=matrix(BASE, BASE, big, 96)) == EINVAL
    assert quantize(L, rows=0, by_rows=matrix(0, 0, 0, 96)) == OK
    assert quantize(L, cols=0, ld=0, by_rows=matrix(0, 0, 64, 0)) == OK


def test_dequantize_refusals(L):
    q = matrix(BASE, BASE + (1 << 20), 64, 96)
    call = lambda q=q, out=BASE + (2 << 20), ld=96, dtype=F16: L.ring_mx4_dequantize(
        ctypes.byref(q) if q is not None else None, out, ld, dtype, None)
    assert call() == ECUDA
    assert call(q=None) == EINVAL and call(out=None) == EINVAL and call(ld=90) == EINVAL and call(dtype=9) == EINVAL
    assert call(out=BASE + 1 + (2 << 20)) == EINVAL and call(out=BASE + 16) == EALIAS
    assert call(q=matrix(0, 0, 0, 5)) == OK


def test_matmul_refusals(L):
    a, b = matrix(BASE, BASE + (1 << 20), 64, 96), matrix(BASE + (2 << 20), BASE + (3 << 20), 40, 96)
    out, res = BASE + (4 << 20), BASE + (5 << 20)

    def call(a=a, b=b, out=out, ld=40, dtype=BF16, res=None, ld_res=40, d=None):
        return L.ring_mx4_matmul(ctypes.byref(a), ctypes.byref(b), out, ld, dtype, res, ld_res, d, None)

    assert call() == ECUDA and call(res=res, d=drop(0.5)) == ECUDA and call(res=out) == ECUDA and call(a=b, out=out) == ECUDA
    assert call(b=matrix(BASE + (2 << 20), BASE + (3 << 20), 40, 95)) == EINVAL
    assert call(out=None) == EINVAL and call(ld=39) == EINVAL and call(dtype=7) == EINVAL and call(out=out + 1) == EINVAL
    assert call(res=res, ld_res=39) == EINVAL and call(res=res + 1) == EINVAL and call(d=drop(1.0)) == EINVAL
    assert call(out=BASE) == EALIAS and call(out=BASE + (3 << 20)) == EALIAS
    assert call(res=out, ld_res=41) == EALIAS and call(res=out + 64) == EALIAS
    assert call(a=matrix(0, 0, 0, 96)) == OK and call(b=matrix(0, 0, 0, 96)) == OK


def test_dropout_refusals(L):
    def call(x=BASE, ldx=64, res=None, ldr=64, out=BASE + (1 << 20), ldo=64, rows=8, cols=64, dtype=F32, d=None):
        return L.ring_dropout(x, ldx, res, ldr, out, ldo, rows, cols, dtype, drop(0.5) if d is None else d, None)

    assert call() == ECUDA and call(out=BASE) == ECUDA and call(res=BASE + (1 << 20)) == ECUDA
    assert L.ring_dropout(BASE, 64, None, 0, BASE + (1 << 20), 64, 8, 64, F32, None, None) == EINVAL
    assert call(x=None) == EINVAL and call(out=BASE + 2 + (1 << 20)) == EINVAL and call(ldx=63) == EINVAL
    assert call(dtype=5) == EINVAL and call(d=drop(1.5)) == EINVAL and call(d=drop(float("nan"))) == EINVAL
    assert call(out=BASE + 64) == EALIAS and call(out=BASE, ldo=65) == EALIAS
    assert call(rows=0) == OK and call(cols=0) == OK
    assert call(rows=1 << 40, cols=1 << 40) == EINVAL


def test_columns_of_one_array_are_no_overlap(L):
    """x or a residual beside the output in the rows of one array, before it and after it; a row that runs into
    the other's columns, or another row pitch, is an overlap still."""
    a, b = matrix(BASE, BASE + (1 << 20), 64, 96), matrix(BASE + (2 << 20), BASE + (3 << 20), 40, 96)
    at = BASE + (4 << 20)

    def product(out, res, ld=100, ld_res=100):
        return L.ring_mx4_matmul(ctypes.byref(a), ctypes.byref(b), out, ld, BF16, res, ld_res, None, None)

    def drops(x, out, res=None, ld=100, ldo=100):
        return L.ring_dropout(x, ld, res, ld, out, ldo, 64, 40, BF16, drop(0.5), None)

    for n in (40, 45, 60):
        for p, q in ((at, at + 2 * n), (at + 2 * n, at), (at, at + 200 + 2 * n), (at + 600 + 2 * n, at)):
            assert product(p, q) == ECUDA and drops(p, q) == ECUDA
            assert drops(BASE, p, res=q) == ECUDA and drops(q, p, res=p) == ECUDA
            assert product(p, q, ld_res=101) == EALIAS and drops(p, q, ldo=101) == EALIAS
    for n in (39, 61, 99, 100, 101):
        for p, q in ((at, at + 2 * n), (at + 2 * n, at), (at, at + 600 + 2 * n), (at + 600 + 2 * n, at)):
            assert product(p, q) == EALIAS and drops(p, q) == EALIAS and drops(BASE, p, res=q) == EALIAS


def test_allreduce_refusals(L):
    from ring_allreduce_reducescatter_gb300 import mx4

    def call(R=3, cols=(96, 96, 96), outs=None, dtype=F32, null=False):
        qs = (mx4._Matrix * max(R, 1))(*[matrix(BASE + (r << 20), BASE + (r << 20) + (1 << 19), 64, cols[r % len(cols)])
                                         for r in range(max(R, 1))])
        outs = outs or [BASE + ((100 + r) << 20) for r in range(max(R, 1))]
        return L.ring_mx4_allreduce(None if null else qs, (ctypes.c_void_p * len(outs))(*outs), R, dtype, None)

    assert call() == ECUDA
    assert call(R=0) == EINVAL and call(R=65) == EINVAL and call(dtype=4) == EINVAL and call(null=True) == EINVAL
    assert call(cols=(96, 95)) == EINVAL
    assert call(outs=[BASE + (100 << 20), 0, BASE + (102 << 20)]) == EINVAL
    assert call(outs=[BASE + (100 << 20)] * 3) == EALIAS
    assert call(outs=[BASE + (100 << 20), BASE + (101 << 20), BASE + 16]) == EALIAS


def test_binding_refuses_host_tensors():
    import torch

    import ring_allreduce_reducescatter_gb300 as rr

    x = torch.zeros((4, 32))
    with pytest.raises(ValueError):
        rr.mx4_quantize(x)
    with pytest.raises(ValueError):
        rr.dropout(x, rr.Dropout(0.1, 0))
    with pytest.raises(ValueError):
        rr.Mx4(torch.zeros(4 * 16, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8), 4, 32)
