"""Attention over a shared prefix, own slots and a call's own rows in 64 bits, with the error bound of the
library's sums: numpy only."""
import numpy as np

U = 2.0 ** -24


def slots(pool, page_table, page, b, n):
    """Slots 0 .. n - 1 of sequence b: [n][Hkv][dh]."""
    if not page:
        return pool[b, :n]
    t = np.arange(n)
    return pool[page_table[b, t // page], t % page]


def attention(q, parts, sees, scale, half):
    """One sequence: q [n1][Hq][dh]; parts: (k, v) [keys][Hkv][dh] that every row sees; sees [n1][m] for the last
    part's keys (None: all parts are seen by all).  Returns o and the bound of the library's error before its
    last rounding: weights of keys are off by eps = error of the score (a dot product of dh terms in
    float: (dh + 4) u sum|q||k| scale, then one subtraction of a reference of like size) + 8 u for the
    exponential and sums of references; normalised sums by twice that; adding n terms up by n u (tensor cores
    may cut: 2 u a term); `half`: half a step of the type that probabilities are held in."""
    n1, Hq, dh = q.shape
    k = np.concatenate([p[0] for p in parts])
    v = np.concatenate([p[1] for p in parts])
    G = Hq // k.shape[1]
    n = len(k)
    m = 0 if sees is None else sees.shape[1]
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(Hq):
        for r in range(n1):
            on = np.ones(n, bool)
            if m:
                on[n - m:] = sees[r]
            if not on.any():
                continue
            kk, vv = k[on, h // G], v[on, h // G]
            s = kk @ q[r, h] * scale
            ds = ((dh + 4) * 2 * U * (np.abs(kk) @ np.abs(q[r, h])) * scale + 2 * U * np.abs(s)).max()
            p = np.exp(s - s.max())
            p /= p.sum()
            o[r, h] = p @ vv
            tol[r, h] = (2 * (ds + 2 * U * np.abs(s).max() + 8 * U) + 2 * (on.sum() + 16) * U + half) * (p @ np.abs(vv))
    return o, tol
