"""The microscaled 4-bit format, the generator and dropout in 64 bits, on the
CPU, for the tests: written from the definitions in include/ringred.h, sharing
nothing with the kernels."""
import numpy as np
import torch

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def philox(seed, sub, group):
    """The four 32-bit words of one counter (plain integers)."""
    c = [group & 0xFFFFFFFF, group >> 32, sub & 0xFFFFFFFF, sub >> 32]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def numbers(seed, sub, first, n):
    """The 16-bit numbers of elements first .. first + n - 1 (numpy, 64-bit words)."""
    g0, g1 = first >> 3, (first + n + 7) >> 3
    m32 = np.uint64(0xFFFFFFFF)
    g = np.uint64(g0) + np.arange(g1 - g0, dtype=np.uint64)
    c0, c1 = g & m32, g >> np.uint64(32)
    c2 = np.full_like(g, sub & 0xFFFFFFFF)
    c3 = np.full_like(g, sub >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p, q = c0 * np.uint64(0xD2511F53), c2 * np.uint64(0xCD9E8D57)
        c0, c1, c2, c3 = ((q >> np.uint64(32)) ^ c1 ^ np.uint64(k0), q & m32,
                          (p >> np.uint64(32)) ^ c3 ^ np.uint64(k1), p & m32)
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    out = np.empty((g.size, 8), dtype=np.int64)
    for j, w in enumerate((c0, c1, c2, c3)):
        out[:, 2 * j], out[:, 2 * j + 1] = w & np.uint64(0xFFFF), w >> np.uint64(16)
    return out.reshape(-1)[first - 8 * g0:first - 8 * g0 + n]


def drop_factor(p, seed, sub, first, rows, cols):
    """0 or 65536 / (65536 - T) for each element; the factor as the library holds it, in binary32."""
    t = int(np.floor(p * 65536 + 0.5))
    u = numbers(seed, sub, first, rows * cols).reshape(rows, cols)
    return np.where(u >= t, np.float64(np.float32(65536 / (65536 - t))), 0.0), u >= t


def quantize(x, random=None):
    """(codes [rows, 32 * blocks], scale bytes [rows, blocks]) of x (binary32 or
    binary64 holding binary32 values), along the last axis; random: (seed, subsequence)."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    neg = np.signbit(b).reshape(rows, nb, 32)
    b = np.abs(b).reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    b[bad] = 0
    neg[bad] = False
    top = b.max(-1)
    m, e = np.frexp(top)  # top = m 2^e, 0.5 <= m < 1
    # 2m <= 1.5: 2^(e - 1) * 2m <= 6 * 2^(e - 3)
    x_exp = np.where(top == 0, -127, np.where(m <= 0.75, e - 3, e - 2))
    x_exp = np.maximum(x_exp, -127)
    v = np.ldexp(b, -x_exp[..., None])
    low = np.clip(np.searchsorted(GRID, v, side="right") - 1, 0, 6)
    f = (v - GRID[low]) / (GRID[low + 1] - GRID[low])
    if random is None:
        up = (f > 0.5) | ((f == 0.5) & (low % 2 == 1))
    else:
        u = numbers(random[0], random[1], 0, rows * nb * 32).reshape(rows, nb, 32)
        up = np.floor(f * 65536) + u >= 65536
    codes = low + up + 8 * neg
    return codes.reshape(rows, nb * 32), np.where(bad, 255, x_exp + 127)


def values(codes, scales, cols):
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales - 127))
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(codes.shape)[:, :cols]


def pack(codes, scales):
    """Stored bytes: data [rows, 16 * blocks], scales [row tiles, column tiles, 1024]."""
    rows, nb = scales.shape
    data = (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)
    tr, tk = -(-rows // 128), -(-nb // 8)
    tiles = np.zeros((tr, tk, 1024), dtype=np.uint8)
    for r in range(rows):
        for j in range(nb):
            tiles[r // 128, j // 8, j // 4 % 2 * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4] = scales[r, j]
    return data, tiles


def unpack(data, tiles, rows, cols):
    nb = -(-cols // 32)
    codes = np.empty((rows, nb * 32), dtype=np.int64)
    codes[:, 0::2], codes[:, 1::2] = data & 15, data >> 4
    r, j = np.arange(rows)[:, None], np.arange(nb)[None, :]
    scales = tiles[r // 128, j // 8, j // 4 % 2 * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4].astype(np.int64)
    return codes, scales


def random_matrix(rows, cols, seed, spread=6):
    """A stored matrix with random codes and scales 2^-spread .. 2^spread:
    (data, tiles) and its values in 64 bits."""
    g = np.random.default_rng(seed)
    nb = -(-cols // 32)
    codes = g.integers(0, 16, (rows, nb * 32))
    codes[:, cols:] = 0
    scales = 127 + g.integers(-spread, spread + 1, (rows, nb))
    data, tiles = pack(codes, scales)
    return torch.from_numpy(data), torch.from_numpy(tiles), values(codes, scales, cols)
