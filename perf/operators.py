"""The microscaled 4-bit operators and dropout as measured cases.

Five kinds of case, each one pass of what a data-parallel training or serving
step does with them:

  quantize  a matrix to microscaled 4 bits (along its rows, its columns or
            both), and back to the values that the 4 bits stand for
  product   out = A B^T of two matrices held in microscaled 4 bits
  dropout   y = residual + dropout(x) and dx = dropout'(dy), mask from a
            counter-based generator
  exchange  the AllReduce of R ranks' gradients on a 4-bit wire: every rank's
            gradient quantised with stochastic rounding, the 4-bit values
            folded in ring order in binary32
  layer     one training step of y = residual + dropout(x W^T) in 4 bits: the
            output and the gradients of x and W

Definitions.  A block is 32 neighbours along the quantised axis (the last one
may be short) with one scale 2^X; X is the smallest integer >= -127 with
max|x| <= 6 * 2^X.  An element is the value of the grid 0, 0.5, 1, 1.5, 2, 3,
4, 6 nearest to |x| / 2^X (ties to the even one of the two grid places), with
x's sign; or, stochastic, with f the way from the grid value below to the one
above, the one above if floor(f * 2^16) + u >= 2^16 for the element's 16-bit
random number u.  Random numbers: Philox4x32-10 (Salmon, Moraes, Dror, Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011) with the seed as key and
(i / 8, subsequence) as counter gives the eight 16-bit numbers of elements i ..
i + 7.  In a quantised matrix, element (r, k) of the result has
i = r * 32 * ceil(K / 32) + k; in dropout i is the row-major index.  Dropout
keeps an element if its number is at least T = round(65536 p) and multiplies
it by 65536 / (65536 - T).
"""
import torch

own = False

BLOCK = 32
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # one token's hidden state before a 4-bit product (serving, batch one)
        dict(name="quantize_token", kind="quantize", rows=1, cols=4096, dtype="bf16", way="rows", rounding="nearest"),
        # a micro-batch of activations, once for the forward product and once for the weight gradient
        dict(name="quantize_activations", kind="quantize", rows=8192, cols=4096, dtype="bf16", way="both", rounding="nearest"),
        # an odd-sized binary32 gradient, transposed and rounded without bias
        dict(name="quantize_odd_gradient", kind="quantize", rows=5003, cols=1999, dtype="f32", way="cols", rounding="stochastic"),
        # decoding one token through the up projection
        dict(name="product_token", kind="product", m=1, n=11008, k=4096, out="bf16"),
        # a small serving batch through the down projection
        dict(name="product_batch_33", kind="product", m=33, n=4096, k=11008, out="f16"),
        # a training micro-batch through the up projection
        dict(name="product_train", kind="product", m=8192, n=11008, k=4096, out="bf16"),
        # residual and dropout of a short prompt
        dict(name="dropout_short", kind="dropout", rows=17, cols=4096, dtype="f16", p=0.1),
        # residual and dropout of a training micro-batch
        dict(name="dropout_train", kind="dropout", rows=16384, cols=4096, dtype="bf16", p=0.1),
        # one projection's gradient over eight ranks
        dict(name="exchange_projection", kind="exchange", ranks=8, rows=4096, cols=4096, dtype="bf16"),
        # a small odd gradient over three ranks
        dict(name="exchange_small", kind="exchange", ranks=3, rows=333, cols=1001, dtype="f32"),
        # a whole training step of one projection
        dict(name="layer_step", kind="layer", m=4096, n=4096, k=4096, p=0.1),
        # the same step with odd sizes in all three directions
        dict(name="layer_odd", kind="layer", m=1003, n=777, k=1537, p=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _bounded(rng, most, *ranges):
    """Sizes of these ranges (over their logarithms) whose product is at most `most`."""
    sizes = [_log(rng, lo, hi) for lo, hi in ranges]
    total = 1
    for s in sizes:
        total *= s
    if total > most:
        big = max(range(len(sizes)), key=lambda j: sizes[j])
        sizes[big] = max(ranges[big][0], sizes[big] * most // total)
    return sizes


def draw(rng):
    kind = rng.choice(("quantize", "product", "product", "dropout", "exchange", "layer"))
    if kind == "quantize":
        rows, cols = _bounded(rng, 8192 * 4096, (1, 16384), (33, 12000))
        return dict(kind=kind, rows=rows, cols=cols, dtype=rng.choice(("f32", "f16", "bf16")),
                    way=rng.choice(("rows", "cols", "both")), rounding=rng.choice(("nearest", "stochastic")))
    if kind == "product":
        m, n, k = _bounded(rng, 8192 * 11008 * 4096, (1, 8192), (64, 11008), (64, 11008))
        return dict(kind=kind, m=m, n=n, k=k, out=rng.choice(("f16", "bf16")))
    if kind == "dropout":
        rows, cols = _bounded(rng, 16384 * 4096, (1, 16384), (33, 12000))
        return dict(kind=kind, rows=rows, cols=cols, dtype=rng.choice(("f32", "f16", "bf16")), p=rng.choice((0.05, 0.1, 0.25, 0.5)))
    if kind == "exchange":
        ranks = rng.randint(2, 8)
        rows, cols = _bounded(rng, 8 * 4096 * 4096 // ranks, (16, 8192), (33, 11008))
        return dict(kind=kind, ranks=ranks, rows=rows, cols=cols, dtype=rng.choice(("f32", "bf16")))
    m, n, k = _bounded(rng, 4096 ** 3, (16, 8192), (64, 8192), (64, 8192))
    return dict(kind=kind, m=m, n=n, k=k, p=rng.choice((0.0, 0.1, 0.2)))


def _mx4_bytes(rows, cols):
    """4-bit elements and one byte of scale for each block."""
    blocks = rows * -(-cols // BLOCK)
    return rows * cols / 2 + blocks


def work(case):
    kind = case["kind"]
    if kind == "quantize":
        n, outs = case["rows"] * case["cols"], 2 if case["way"] == "both" else 1
        return {"bytes": n * SIZE[case["dtype"]] + outs * n * 2, "flops": 0}
    if kind == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _mx4_bytes(m, k) + _mx4_bytes(n, k) + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    if kind == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": 5 * n * SIZE[case["dtype"]], "flops": 0}
    if kind == "exchange":
        n = case["ranks"] * case["rows"] * case["cols"]
        return {"bytes": 2 * n * SIZE[case["dtype"]], "flops": n}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": 2 * (2 * m * k + 2 * n * k + 3 * m * n), "flops": 6 * m * n * k}


# ----------------------------------------------------------------- the inputs


def _normal(g, shape, sigma, dtype):
    return torch.randn(shape, generator=g, device="cuda").mul_(sigma).to(dtype)


def _activations(g, rows, cols, dtype):
    """Activations with a few columns far larger than the others, as hidden states have."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    loud = (torch.rand((1, cols), generator=g, device="cuda") < 0.01).float()
    return (x * (1 + 15 * loud)).to(dtype)


def _pack(codes, x):
    """The stored form of grid places (rows, K32) with sign and exponents x (rows, K32 / 32): two
    elements a byte, the lower one in the low half; scale bytes x + 127 in tiles of 128 rows and 8
    blocks, the tile's byte (r % 32) * 16 + r / 32 * 4 + j % 4 of its half j / 4 for row r, block j."""
    data = (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8)
    rows, blocks = x.shape
    tr, tk = -(-rows // 128), -(-blocks // 8)
    full = torch.zeros((tr * 128, tk * 8), dtype=torch.uint8, device=x.device)
    full[:rows, :blocks] = (x + 127).to(torch.uint8)
    tiles = full.view(tr, 4, 32, tk, 2, 4).permute(0, 3, 4, 2, 1, 5).contiguous()
    return data.contiguous(), tiles.view(tr, tk, 1024)


def _unpack(data, scales, rows, cols):
    """The binary32 values of a stored matrix."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=data.device)
    d = data.long()
    v = grid[torch.stack((d & 15, d >> 4), -1).view(rows, -1)]
    tr, tk = scales.shape[0], scales.shape[1]
    full = scales.view(tr, tk, 2, 32, 4, 4).permute(0, 4, 3, 1, 2, 5).reshape(tr * 128, tk * 8)
    x = full[:rows, :v.shape[1] // BLOCK].to(torch.int32) - 127
    return (v.view(rows, -1, BLOCK) * _power(x).unsqueeze(-1)).view(rows, -1)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, s = case["kind"], dict(case)
    s["seed"], s["sub"] = 0x9E3779B97F4A7C15 * (int(seed) + 1) & (1 << 63) - 1, int(seed) * 16
    if kind == "quantize":
        t = TYPES[case["dtype"]]
        s["x"] = (_activations(g, case["rows"], case["cols"], t) if case["rounding"] == "nearest"
                  else _normal(g, (case["rows"], case["cols"]), 1e-3, t))
    elif kind == "product":
        for name, rows, scale in (("a", case["m"], 1.0), ("b", case["n"], 0.02)):
            x = _activations(g, rows, case["k"], torch.float32) if name == "a" else _normal(g, (rows, case["k"]), scale, torch.float32)
            codes, e = _codes(x, None)
            s[name] = _pack(codes, e)
    elif kind == "dropout":
        t, shape = TYPES[case["dtype"]], (case["rows"], case["cols"])
        s["x"], s["residual"], s["dy"] = (_normal(g, shape, sigma, t) for sigma in (1.0, 1.0, 1e-2))
    elif kind == "exchange":
        t = TYPES[case["dtype"]]
        s["grads"] = [_normal(g, (case["rows"], case["cols"]), 1e-3, t) for _ in range(case["ranks"])]
    else:
        m, n, k, t = case["m"], case["n"], case["k"], torch.bfloat16
        s["x"], s["w"] = _activations(g, m, k, t), _normal(g, (n, k), 0.02, t)
        s["residual"], s["dy"] = _normal(g, (m, n), 1.0, t), _normal(g, (m, n), 1e-2, t)
    return s


# ------------------------------------------------------------ the plain forms


def _power(x):
    """2^x in binary32 for whole x in -127 .. 127."""
    bits = torch.where(x > -127, (x + 127) << 23, 1 << 22)
    return bits.to(torch.int32).view(torch.float32)


def _philox(seed, sub, groups):
    """The eight 16-bit random numbers of each counter in `groups` (int64), last axis 8."""
    c0, c1 = groups & M32, groups >> 32
    c2, c3 = torch.full_like(groups, sub & M32), torch.full_like(groups, sub >> 32)
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & M32) ^ c1 ^ k0, p1 & M32, (p0 >> 32 & M32) ^ c3 ^ k1, p0 & M32
        k0, k1 = k0 + 0x9E3779B9 & M32, k1 + 0xBB67AE85 & M32
    words = torch.stack((c0, c1, c2, c3), -1)
    return torch.stack((words & 0xFFFF, words >> 16), -1).flatten(-2)


def _numbers(seed, sub, n, device):
    """The random numbers of elements 0 .. n - 1."""
    groups = torch.arange(-(-n // 8), dtype=torch.int64, device=device)
    return _philox(seed, sub, groups).view(-1)[:n]


def _blocks(x):
    """(rows, K) in binary32 as (rows, blocks, 32), padded with zeros, and every block's exponent."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    x = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m == 0, -127, torch.where(m <= 0.75, e - 3, e - 2)).clamp_(min=-127)
    return x, e.to(torch.int32)


def _places(x, e, random):
    """Grid places 0 .. 7 of |x| / 2^e; random: None (nearest), or (seed, subsequence)."""
    v = x.abs() * _power(-e).unsqueeze(-1)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    t = v / step
    if random is None:
        t = torch.round(t)
    else:
        low = torch.floor(t)
        u = _numbers(*random, x.numel(), x.device).view(x.shape)
        t = low + (torch.floor((t - low) * 65536) + u >= 65536)
    return (t + torch.where(v < 2, 0, torch.where(v < 4, 2, 4))).to(torch.int64)


def _codes(x, random):
    b, e = _blocks(x)
    return (_places(b, e, random) + 8 * (b < 0)).view(b.shape[0], -1), e


def _rounded(x, random):
    """The values of x after quantisation along its last axis, in binary32."""
    b, e = _blocks(x)
    grid = torch.tensor(GRID, device=x.device)
    v = grid[_places(b, e, random)]
    return (torch.where(b < 0, -v, v) * _power(e).unsqueeze(-1)).view(b.shape[0], -1)[:, :x.shape[1]]


def _kept(p, seed, sub, shape, device):
    """0 for a dropped element, 1 / (1 - p) for a kept one."""
    n = shape[0] * shape[1]
    t = int(p * 65536 + 0.5)
    u = _numbers(seed, sub, n, device).view(shape)
    return (u >= t).float() * (65536 / (65536 - t))


def _ring_sum(vs):
    """The ring's fold of R equal matrices: chunk c of the flat index starts at rank c."""
    ranks, n = len(vs), vs[0].numel()
    v = torch.stack([x.reshape(-1) for x in vs])
    at = torch.arange(n, device=v.device)
    chunk = (at // max(n // ranks, 1)).clamp_(max=ranks - 1) if n >= ranks else torch.full_like(at, ranks - 1)
    total = v[chunk, at]
    for step in range(1, ranks):
        total = total + v[(chunk + step) % ranks, at]
    return total.view(vs[0].shape)


def _plain(s):
    kind, seed, sub = s["kind"], s["seed"], s["sub"]
    if kind == "quantize":
        stochastic = s["rounding"] == "stochastic"
        outs = {}
        if s["way"] != "cols":
            outs["rows"] = _rounded(s["x"], (seed, sub) if stochastic else None).to(torch.bfloat16)
        if s["way"] != "rows":
            outs["cols"] = _rounded(s["x"].t().contiguous(), (seed, sub + 1) if stochastic else None).to(torch.bfloat16)
        return outs
    if kind == "product":
        a, b = _unpack(*s["a"], s["m"], s["k"]), _unpack(*s["b"], s["n"], s["k"])
        return (a @ b.t()).to(TYPES[s["out"]])
    if kind == "dropout":
        d = _kept(s["p"], seed, sub, s["x"].shape, s["x"].device)
        t = TYPES[s["dtype"]]
        return {"y": (s["residual"].float() + s["x"].float() * d).to(t), "dx": (s["dy"].float() * d).to(t)}
    if kind == "exchange":
        y = _ring_sum([_rounded(x, (seed, sub + r)) for r, x in enumerate(s["grads"])]).to(TYPES[s["dtype"]])
        return [y.clone() for _ in s["grads"]]
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    d = _kept(s["p"], seed, sub, dy.shape, dy.device)
    y = s["residual"].float() + (_rounded(x, None) @ _rounded(w, None).t()) * d
    g = dy * d
    dx = _rounded(g, (seed, sub + 1)) @ _rounded(w.t().contiguous(), None).t()
    dw = _rounded(g.t().contiguous(), (seed, sub + 2)) @ _rounded(x.t().contiguous(), None).t()
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


# ------------------------------------------------------- the framework's calls


def _own(s):
    import ring_allreduce_reducescatter_gb300 as rr

    kind, seed, sub = s["kind"], s["seed"], s["sub"]
    if kind == "quantize":
        how = dict(rounding=s["rounding"], seed=seed, subsequence=sub)
        if s["way"] == "both":
            rows, cols = rr.mx4_quantize_both(s["x"], **how)
            return {"rows": rr.mx4_dequantize(rows, torch.bfloat16), "cols": rr.mx4_dequantize(cols, torch.bfloat16)}
        if s["way"] == "rows":
            return {"rows": rr.mx4_dequantize(rr.mx4_quantize(s["x"], **how), torch.bfloat16)}
        how["subsequence"] = sub + 1
        return {"cols": rr.mx4_dequantize(rr.mx4_quantize(s["x"], transposed=True, **how), torch.bfloat16)}
    if kind == "product":
        a, b = rr.Mx4(*s["a"], s["m"], s["k"]), rr.Mx4(*s["b"], s["n"], s["k"])
        return rr.mx4_matmul(a, b, TYPES[s["out"]])
    if kind == "dropout":
        d = rr.Dropout(s["p"], seed, sub)
        return {"y": rr.dropout(s["x"], d, residual=s["residual"]), "dx": rr.dropout(s["dy"], d)}
    if kind == "exchange":
        qs = [rr.mx4_quantize(x, rounding="stochastic", seed=seed, subsequence=sub + r) for r, x in enumerate(s["grads"])]
        return rr.mx4_allreduce(qs, dtype=TYPES[s["dtype"]])
    d = rr.Dropout(s["p"], seed, sub)
    x_rows, x_cols = rr.mx4_quantize_both(s["x"])
    w_rows, w_cols = rr.mx4_quantize_both(s["w"])
    y = rr.mx4_matmul(x_rows, w_rows, torch.bfloat16, residual=s["residual"], dropout=d)
    g_rows, g_cols = rr.mx4_quantize_both(s["dy"], rounding="stochastic", seed=seed, subsequence=sub + 1, dropout=d)
    return {"y": y, "dx": rr.mx4_matmul(g_rows, w_cols, torch.bfloat16), "dw": rr.mx4_matmul(g_cols, x_cols, torch.bfloat16)}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------- the definition in 64 bits


def _exact_numbers(seed, sub, n, device):
    """Philox4x32-10 with its products taken in 16-bit halves, 16 bits a number."""
    i = torch.arange((n + 7) // 8, dtype=torch.int64, device=device)

    def product(c, m):
        low, high = c * (m % 65536), c * (m // 65536)
        mid = high + low // 65536
        return mid // 65536, mid % 65536 * 65536 + low % 65536

    a, b = i % 2 ** 32, i // 2 ** 32
    c = torch.zeros_like(i) + sub % 2 ** 32
    d = torch.zeros_like(i) + sub // 2 ** 32
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for r in range(10):
        k = (key[0] + r * 0x9E3779B9) % 2 ** 32, (key[1] + r * 0xBB67AE85) % 2 ** 32
        (ha, la), (hc, lc) = product(a, 0xD2511F53), product(c, 0xCD9E8D57)
        a, b, c, d = torch.bitwise_xor(torch.bitwise_xor(hc, b), k[0]), lc, torch.bitwise_xor(torch.bitwise_xor(ha, d), k[1]), la
    out = torch.empty((i.numel(), 8), dtype=torch.int32, device=device)
    for j, w in enumerate((a, b, c, d)):
        out[:, 2 * j], out[:, 2 * j + 1] = w % 65536, w // 65536
    return out.view(-1)[:n]


def _exact_rounded(x, random=None):
    """x (64 bits) after quantisation along its last axis, by comparison with the grid's values."""
    rows, cols = x.shape
    nb = (cols + 31) // 32
    full = torch.zeros((rows, nb * 32), dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    u = None if random is None else _exact_numbers(*random, full.numel(), x.device).view(rows, nb * 32)
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    out = torch.empty_like(full)
    part = max(1, (1 << 24) // (nb * 32))
    for r in range(0, rows, part):
        b = full[r:r + part].view(-1, nb, 32)
        top = b.abs().max(-1, keepdim=True).values / 6
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140))).clamp(min=-127)
        e = torch.where(torch.exp2(e - 1) >= top, e - 1, torch.where(torch.exp2(e) < top, e + 1, e)).clamp(min=-127)
        v = (b.abs() / torch.exp2(e)).contiguous()
        low = (torch.bucketize(v, grid, right=True) - 1).clamp(max=6)
        f = (v - grid[low]) / (grid[low + 1] - grid[low])
        if u is None:
            up = (f > 0.5) | (f == 0.5) & (low % 2 == 1)
        else:
            up = torch.floor(f * 65536) + u[r:r + part].view(b.shape) >= 65536
        out[r:r + part] = (torch.sign(b) * grid[low + up] * torch.exp2(e)).view(-1, nb * 32)
    return out[:, :cols]


def _exact_kept(p, seed, sub, shape, device):
    t = int(p * 65536 + 0.5)
    keep = _exact_numbers(seed, sub, shape[0] * shape[1], device).view(shape) >= t
    return keep.double() / (1 - t / 65536)


def exact(case, seed):
    s = prepare(case, seed)
    kind, key, sub = s["kind"], s["seed"], s["sub"]
    if kind == "quantize":
        some, x, outs = s["rounding"] == "stochastic", s["x"].double(), {}
        if s["way"] in ("rows", "both"):
            outs["rows"] = _exact_rounded(x, (key, sub) if some else None)
        if s["way"] in ("cols", "both"):
            outs["cols"] = _exact_rounded(x.t().contiguous(), (key, sub + 1) if some else None)
        return outs
    if kind == "product":
        sides = []
        for name, rows in (("a", s["m"]), ("b", s["n"])):
            data, scales = s[name]
            blocks = data.shape[1] // 16
            r = torch.arange(rows, device=data.device).view(-1, 1)
            j = torch.arange(blocks, device=data.device).view(1, -1)
            at = ((r // 128 * scales.shape[1] + j // 8) * 1024 + j // 4 % 2 * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4)
            e = scales.reshape(-1)[at].double() - 127
            nibbles = torch.empty((rows, 2 * data.shape[1]), dtype=torch.int64, device=data.device)
            nibbles[:, 0::2], nibbles[:, 1::2] = data % 16, data // 16
            size = torch.tensor(GRID, dtype=torch.float64, device=data.device)[nibbles % 8]
            v = torch.where(nibbles >= 8, -size, size).view(rows, blocks, 32) * torch.exp2(e).unsqueeze(-1)
            sides.append(v.view(rows, -1)[:, :s["k"]])
        return torch.einsum("mk,nk->mn", *sides)
    if kind == "dropout":
        d = _exact_kept(s["p"], key, sub, s["x"].shape, s["x"].device)
        return {"y": torch.addcmul(s["residual"].double(), d, s["x"].double()), "dx": d * s["dy"].double()}
    if kind == "exchange":
        total = sum(_exact_rounded(x.double(), (key, sub + r)) for r, x in enumerate(s["grads"]))
        return [total] * len(s["grads"])
    x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
    d = _exact_kept(s["p"], key, sub, dy.shape, dy.device)
    y = torch.einsum("mk,nk->mn", _exact_rounded(x), _exact_rounded(w)) * d + s["residual"].double()
    g = dy * d
    dx = torch.einsum("mn,kn->mk", _exact_rounded(g, (key, sub + 1)), _exact_rounded(w.t().contiguous()))
    dw = torch.einsum("nm,km->nk", _exact_rounded(g.t().contiguous(), (key, sub + 2)), _exact_rounded(x.t().contiguous()))
    return {"y": y, "dx": dx, "dw": dw}
