"""Plain 64-bit forms of the rotary and cache operators (numpy), for the tests.

A 4-bit cache is handled as its bytes: blocks of 9*dh bytes for 16 slots of one head (see
include/medusa.h), decoded and encoded here from the definitions of e2m1 and e4m3."""
import math

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])
_B = np.arange(256)
_E, _M = (_B >> 3) & 15, _B & 7
E4M3 = np.where(_E > 0, (8 + _M) * 2.0 ** (_E - 10.0), _M * 2.0 ** -9) * np.where(_B >= 128, -1, 1)
E4M3[(_B & 127) == 127] = np.nan


def frequencies(rot, base=10000.0, scaling="plain", factor=1.0, orig_pos=0, low=1.0, high=32.0, **_):
    th = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "plain":
        return th
    if scaling == "linear":
        return th / factor
    if scaling == "banded":
        w = (orig_pos * th / (2 * math.pi) - low) / (high - low)
    else:
        def c(r):
            return rot * math.log(orig_pos / (2 * math.pi * r)) / (2 * math.log(base))
        a, b = max(0, math.floor(c(high))), min(rot - 1, math.ceil(c(low)))
        w = 1 - (np.arange(rot // 2) - a) / max(b - a, 0.001)
    w = np.clip(w, 0, 1)
    return w * th + (1 - w) * th / factor


def rope(x, pos, rot, layout="half", attn=1.0, inverse=False, **kw):
    """x [rows][heads][dh] float64 turned at integer positions pos [rows]."""
    a = np.asarray(pos, dtype=np.float64)[:, None] * frequencies(rot, **kw)
    c, s = (np.cos(a) * attn)[:, None], (np.sin(a) * attn)[:, None]
    s = -s if inverse else s
    y = x.copy()
    i, j = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
            else (slice(0, rot, 2), slice(1, rot, 2)))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def decode(codes, scales, g):
    """codes [..., dh/2], scales [..., dh/16] bytes -> float64 [..., dh]."""
    v = np.stack((E2M1[codes & 15], E2M1[codes >> 4]), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return v * np.repeat(E4M3[scales], 16, -1) * g


def e4m3_nearest(x):
    """Byte of the nearest e4m3 to x >= 0 (ties to even, 448 at most)."""
    grid = E4M3[:127]
    i = np.clip(np.searchsorted(grid, x), 1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 0))
    return np.where(up, i, i - 1).astype(np.uint8)


def e2m1_nearest(a):
    """Code of the nearest e2m1 magnitude to a >= 0, ties to the even code."""
    mid = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])
    lo, hi = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    return np.where(lo % 2 == 0, lo, hi)


def encode(x, g):
    """float64 [..., dh] -> (codes [..., dh/2], scales [..., dh/16])."""
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    s8 = e4m3_nearest(np.abs(y).max(-1) / (6 * g))
    s = (E4M3[s8] * g)[..., None]
    c = np.where(s > 0, e2m1_nearest(np.abs(y) / np.where(s > 0, s, 1)), 0)
    c = (c + 8 * (y < 0)).reshape(x.shape).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), s8


class Pool:
    """A cache's bytes or elements seen slot by slot: where slot t of sequence b lies."""

    def __init__(self, fmt, B, Hkv, dh, capacity, page_size=0, table=None):
        self.fmt, self.B, self.Hkv, self.dh = fmt, B, Hkv, dh
        self.capacity, self.page, self.table = capacity, page_size, table

    def unit(self, b, t):
        if not self.page:
            return b, t
        return int(self.table[b, t // self.page]), t % self.page

    def slot(self, pool, b, t):
        """(codes [Hkv][dh/2], scales [Hkv][dh/16]) views of a 4-bit pool (uint8, flat), or
        the [Hkv][dh] view of a plain one."""
        u, i = self.unit(b, t)
        per = self.page or self.capacity
        if self.fmt != "kv4":
            return pool.reshape(-1, per, self.Hkv, self.dh)[u, i]
        blk = pool.reshape(-1, self.Hkv, per // 16, 9 * self.dh)[u, :, i // 16]
        dh, r = self.dh, i % 16
        return (blk[:, r * dh // 2:(r + 1) * dh // 2],
                blk[:, 8 * dh + r * dh // 16:8 * dh + (r + 1) * dh // 16])

    def value(self, pool, b, t, g=1.0):
        if self.fmt != "kv4":
            return self.slot(pool, b, t).astype(np.float64)
        return decode(*self.slot(pool, b, t), g)

    def prefix(self, pool, b, n, g=1.0):
        """[n][Hkv][dh] float64: what the first n slots of sequence b hold."""
        if n == 0:
            return np.zeros((0, self.Hkv, self.dh))
        return np.stack([self.value(pool, b, t, g) for t in range(n)])


def attention(q, K, V, tk, tv, see, scale):
    """One sequence: q [n1][Hq][dh], K, V [L][Hkv][dh], tk, tv [n1][Hkv][dh] or None, see
    [n1][n1] bool.  Returns (o, spread, reach): spread = sum p |v| and reach = the largest
    scale * sum |q||k| of a visible key, which error bounds are made of."""
    n1, Hq, dh = q.shape
    G = Hq // K.shape[1]
    if tk is not None:
        K, V = np.concatenate((K, tk)), np.concatenate((V, tv))
        vis = np.concatenate((np.ones((n1, len(K) - n1), bool), see), 1)
    else:
        vis = np.ones((n1, len(K)), bool)
    o, spread, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n1, Hq, 1))
    for h in range(Hq):
        k, v = K[:, h // G], V[:, h // G]
        for n in range(n1):
            w = vis[n]
            if not w.any():
                continue
            s = scale * (k[w] @ q[n, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            o[n, h], spread[n, h] = p @ v[w], p @ np.abs(v[w])
            reach[n, h] = scale * (np.abs(k[w]) @ np.abs(q[n, h])).max()
    return o, spread, reach
