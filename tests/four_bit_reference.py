"""Plain 64-bit forms of the 4-bit rows of a paged cache, of the position rotation and of the attention over
selected blocks, in numpy, for the tests: written from the formulas."""
import numpy as np

import dense_reference as ref

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nearest(grid, x):
    """Index of the value of an ascending grid nearest to x >= 0, ties to the even index, clamped to the last."""
    hi = np.clip(np.searchsorted(grid, x), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where(x >= grid[-1], len(grid) - 1, np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi))


def encode_row(x):
    """(codes 0 .. 15, scale bytes, exponent) of one row of d values: the least e in [-100, 100] with
    max|x| <= 2688 * 2^e over the finite values; for each 16 values the e4m3 scale nearest to a sixth of their
    largest over 2^e, and the nearest codes, ties to even.  Sixteen values with an infinity or NaN: a NaN scale."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    top = np.abs(x[fine]).max() if fine.any() else 0.0
    e = -100
    while e < 100 and top > 2688.0 * 2.0 ** e:
        e += 1
    y = (np.where(fine, x, 0.0) * 2.0 ** -e).reshape(-1, 16)
    scales = nearest(ref.e4m3_values()[:127], np.abs(y).max(-1) / 6.0).astype(np.uint8)
    s = ref.e4m3_values()[scales]
    ratio = np.abs(y) / np.where(s > 0, s, 1.0)[:, None]
    codes = nearest(CODES, ratio) + 8 * np.signbit(y)
    whole = fine.reshape(-1, 16).all(-1)
    codes = np.where((whole & (s > 0))[:, None], codes, 0).astype(np.uint8)
    return codes.reshape(-1), np.where(whole, scales, 0x7f).astype(np.uint8), e


def values(codes, scales, exps):
    """codes [..][d], scale bytes [..][d / 16], exponent bytes [..] as 64-bit values."""
    v = CODES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.repeat(ref.e4m3_values()[scales], 16, axis=-1)
    return v * s * 2.0 ** (np.asarray(exps, float) - 127)[..., None]


def unpack(bytes_):
    """Codes of packed bytes [..][d / 2]: the even value is the low half."""
    return np.stack([bytes_ & 15, bytes_ >> 4], -1).reshape(*bytes_.shape[:-1], 2 * bytes_.shape[-1])


def rotate(x, pos, rot, base):
    """x [n][H][d]: values i and i + rot / 2 turned by pos * base^(-2 i / rot), as complex numbers."""
    y = np.array(x, np.float64)
    if rot:
        angle = np.asarray(pos, np.longdouble)[:, None] * np.longdouble(base) ** (-np.arange(rot // 2, dtype=np.longdouble) * 2 / rot)
        turn = np.exp(1j * np.remainder(angle, 2 * np.longdouble("3.14159265358979323846264338327950288")).astype(np.float64))
        z = (y[..., :rot // 2] + 1j * y[..., rot // 2:rot]) * turn[:, None]
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def listed_cells(blocks, count, p):
    """Cells that a token at position p sees: its listed blocks that are complete, and its open block."""
    cells = [4 * int(b) + i for b in blocks[:max(0, count)] if b >= 0 and 4 * int(b) + 3 <= p for i in range(4)]
    return np.array(cells + list(range((p + 1) // 4 * 4, p + 1)), np.int64)
