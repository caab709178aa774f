"""The 8-bit format and its products in 64 bits, from include/medusa.h's description, written apart from the
library: numpy only."""
import numpy as np

G = 128


def decode(c):
    """e4m3 codes (uint8) as numbers."""
    c = np.asarray(c, np.uint8).astype(np.int64)
    m, e = c & 7, (c >> 3) & 15
    v = np.where(e > 0, np.ldexp(8.0 + m, e - 10), np.ldexp(m.astype(float), -9))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c > 127, -v, v)


_ALL = decode(np.arange(127))                       # ascending


def encode(x):
    """Nearest codes of |x| <= 448, ties to even codes."""
    a = np.abs(x)
    i = np.clip(np.searchsorted(_ALL, a), 1, 126)
    lo, hi = _ALL[i - 1], _ALL[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    c = np.where(up, i, i - 1).astype(np.uint8)
    return np.where(np.signbit(x), c | 128, c).astype(np.uint8)


def blocks(x, block):
    """[rows/block][k/128] lists of slices."""
    for i in range(-(-x.shape[0] // block)):
        for j in range(-(-x.shape[1] // G)):
            yield i, j, np.s_[i * block:(i + 1) * block, j * G:(j + 1) * G]


def round8(x, block):
    """Codes and scales of x [rows][k] in 64 bits."""
    codes = np.zeros(x.shape, np.uint8)
    scales = np.zeros((-(-x.shape[0] // block), -(-x.shape[1] // G)))
    for i, j, at in blocks(x, block):
        top = np.abs(x[at]).max()
        if not np.isfinite(top):
            codes[at], scales[i, j] = 127, 1.0
            continue
        s = 1.0
        if top > 0:
            e = -126
            while top > 448 * 2.0 ** e:
                e += 1
            s = 2.0 ** e
        codes[at], scales[i, j] = encode(x[at] / s), s
    return codes, scales


def values(codes, scales, block):
    v = decode(codes)
    s = np.repeat(np.repeat(np.asarray(scales, float), block, 0)[:v.shape[0]], G, 1)[:, :v.shape[1]]
    return v * s


def silu(a):
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a))
