"""Plain 64-bit forms of the operators of an FFN in 8-bit floating point, in
numpy, and bounds of what the kernels' sums may be off by.

Bounds.  With P the sum of |products| of a result (scales included), u = 2^-24:
 - sums in fp32 on the bf16 matrix unit: an instruction adds 32 products, each
   of which may lose a unit of the last place of the largest (2u of it), to the
   running sum, which is rounded once (2u at most): (32 + instructions) * 2u * P,
   the largest product of an instruction being at most its part of P;
 - a block's scale is a rounded product, its FMA rounds, the waves' sums are
   added, the bias too: (2 + blocks + 16 + 1) * 2u * P;
 - on the E4M3 unit products are aligned in eights of neighbouring k and lose
   less than 2^-13 of the largest one's power of two each: 8 * 2^-13 of the sum
   of the eights' largest.
A rounding to bf16 is 2^-8 of the value at most."""
import numpy as np

U = 2.0 ** -24
BLOCK = 128
WIDEST = 448.0


def e4m3_table():
    """Values of the 256 codes."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


TABLE = e4m3_table()


def decode(codes):
    return TABLE[np.asarray(codes, np.uint8)]


def encode(v):
    """Codes of values up to 448, to nearest, ties to even."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    grid = TABLE[:127]
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (c + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def blocks(n):
    return -(-n // BLOCK)


def spread(s, n):
    """A scale for each block of 128 along the last axis, as one for each of n values."""
    return np.repeat(np.asarray(s, np.float64), BLOCK, axis=-1)[..., :n]


def block_max(v):
    T, K = v.shape
    a = np.zeros((T, blocks(K) * BLOCK))
    a[:, :K] = np.abs(v)
    return a.reshape(T, -1, BLOCK).max(axis=2)


def quant(v):
    """The rule of moe_quant_fp8 in its fp32 steps for fp32 values: bits are defined."""
    v = np.asarray(v, np.float32)
    a = block_max(v).astype(np.float32)
    with np.errstate(all="ignore"):
        s = a / np.float32(448)
        pre = np.where(a < 2.0 ** -96, np.float32(2.0 ** 64), np.float32(1))
        inv = np.where(a > 0, np.float32(448) / (a * pre), np.float32(0))
        fine = np.isfinite(a)
        s, inv = np.where(fine, s, np.nan).astype(np.float32), np.where(fine, inv, 0).astype(np.float32)
        wide = lambda x: np.repeat(x, BLOCK, axis=1)[:, :v.shape[1]]  # noqa: E731
        p = np.where(wide(inv) == 0, np.float32(0), (v * wide(pre).astype(np.float32)) * wide(inv))
    return encode(p), s


def scaled(codes, s):
    """The values that codes [n, K] with scales [n, ceil(K/128)] stand for."""
    return decode(codes) * spread(s, codes.shape[-1])


def scaled_weights(w, ws):
    """The same for weights [.., N, K] with scales [.., ceil(N/128), ceil(K/128)]."""
    N, K = w.shape[-2:]
    return decode(w) * spread(np.repeat(np.asarray(ws, np.float64), BLOCK, axis=-2)[..., :N, :], K)


def eights(x, w):
    """Sum over eights of neighbouring k of the largest |x*w|, [T, N]."""
    T, K = x.shape
    pad = -K % 8
    x = np.pad(np.abs(x), ((0, 0), (0, pad))).reshape(T, -1, 8)
    w = np.pad(np.abs(w), ((0, 0), (0, pad))).reshape(w.shape[0], -1, 8)
    out = np.zeros((T, w.shape[0]))
    for t in range(T):
        out[t] = (x[t][None] * w).max(axis=2).sum(axis=1)
    return out


def limit(x, w, size, out_bf16, unit_fp8):
    """What a product of values x [T,K], w [N,K] may be off by, [T,N]; size: bytes of a value in memory."""
    K = x.shape[1]
    P = np.abs(x) @ np.abs(w).T
    lim = (32 + K / 32 + 4 * blocks(K) + 19 + blocks(K * size)) * 2 * U * P
    if unit_fp8:
        lim += 8 * 2.0 ** -13 * eights(x, w)
    if out_bf16:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(x @ w.T)
    return lim + 1e-37


def some_rows(n, first=0):
    """Up to some 40 of n rows: those around the tiles' borders, and a few between."""
    if n <= 40:
        return np.arange(first, first + n)
    edges = [r + d for r in (0, 16, 32, 64, 128, 192, 256, n) for d in (-1, 0)] + [r for r in (n // 3, n // 2, n - 17, n - 33)]
    edges += list(range(0, n, max(1, n // 16)))
    return first + np.unique([r for r in edges if 0 <= r < n])


def group(idx, E):
    """offsets, rows, pos of ids [T,k]."""
    flat = np.asarray(idx).reshape(-1)
    ok = (flat >= 0) & (flat < E)
    where = np.flatnonzero(ok)
    order = where[np.argsort(flat[where], kind="stable")]
    offsets = np.zeros(E + 1, np.int32)
    np.cumsum(np.bincount(flat[where], minlength=E), out=offsets[1:])
    pos = np.full(flat.size, -1, np.int32)
    pos[order] = np.arange(order.size)
    return offsets, (order // np.asarray(idx).shape[1]).astype(np.int32), pos.reshape(np.asarray(idx).shape)


def codes(r, *shape):
    """Codes of normal values, their largest near 448."""
    return encode(np.clip(r.standard_normal(shape) * 150, -WIDEST, WIDEST))
