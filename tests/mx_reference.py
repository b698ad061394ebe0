"""The 4-bit microscaled formats in fp64 numpy, from their definition: block
scales, E2M1 rounding, the tiled scale layout and the products.  Test side
only; shares no code with the library."""
import numpy as np

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    v = []
    for b in range(127):  # 0x7f is NaN
        e, m = b >> 3, b & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3 = e4m3_values()


def _nearest_even(x, grid):
    """Index of the grid value (ascending, from 0) nearest to x >= 0; a tie goes
    to the even index, past the end to the last."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, x, side="left")   # mids < x
    hi = np.searchsorted(mid, x, side="right")  # mids <= x
    return np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))


def quantize(X, fmt, factor=1.0):
    """(codes 0..15 [rows, K], scale bytes [rows, blocks]) of the rows of X."""
    X = np.asarray(X, dtype=np.float64)
    rows, K = X.shape
    b = BLOCK[fmt]
    n = -(-K // b)
    P = np.zeros((rows, n * b))
    P[:, :K] = X
    P = P.reshape(rows, n, b)
    amax = np.abs(P).max(-1)
    bad = ~np.isfinite(P).all(-1)
    amax = np.where(bad, 1.0, amax)
    if fmt == MX:
        _, e = np.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1
        byte = np.where(amax > 0, np.clip(e - 1 - 2, -127, 127) + 127, 0)
        unit = np.exp2(byte - 127.0)
    else:
        f = np.float64(np.float32(factor))
        byte = _nearest_even(np.minimum(amax / (6 * f), 448.0), E4M3)
        unit = E4M3[byte] * f
    byte = np.where(bad, 0xFF if fmt == MX else 0x7F, byte)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(unit[..., None] > 0, P / np.where(unit > 0, unit, 1)[..., None], 0.0)
    t = np.where(bad[..., None], 0.0, t)
    code = _nearest_even(np.abs(t), LEVELS) + 8 * np.signbit(P)
    return code.reshape(rows, n * b)[:, :K].astype(np.uint8), byte.astype(np.uint8)


def dequantize(codes, bytes_, fmt, factor=1.0):
    rows, K = codes.shape
    v = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    b = BLOCK[fmt]
    if fmt == MX:
        s = np.where(bytes_ == 0xFF, np.nan, np.exp2(bytes_.astype(np.float64) - 127))
    else:
        s = np.where(bytes_ == 0x7F, np.nan, E4M3[np.minimum(bytes_, 126)]) * np.float64(np.float32(factor))
    return v * np.repeat(s, b, axis=1)[:, :K]


def unpack_codes(packed, K):
    """(rows, row_bytes) uint8 to codes (rows, K): the even value in the low half."""
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out[:, :K]


def untile_scales(flat, rows, K, fmt):
    """Tiled scale bytes to (rows, blocks)."""
    n = -(-K // BLOCK[fmt])
    tiles = -(-n // 4)
    r, s = np.meshgrid(np.arange(rows), np.arange(n), indexing="ij")
    return flat[((r // 128) * tiles + s // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + s % 4]


def product_bound(A, B, K):
    """How far fp32 accumulation may be from sum_k a b: the products are exact,
    and K of them are added in groups of 64; each addition into the running
    sum, and the sum within a group, is allowed two units in the last place of
    what has been added in magnitude."""
    return (K / 64 + 8) * 2.0 ** -22 * (np.abs(A) @ np.abs(B).T)
