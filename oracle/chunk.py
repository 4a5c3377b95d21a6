"""Oracle of the operators in include/qsa_rope.h and include/qsa_chunk.h: norms
with rotation, attention of ragged chunks, attention behind a shared prefix.

Plain numpy in binary64 and Python integers, from the headers' definitions.
Shares nothing with the CUDA library.  Inputs come as the values they hold."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .cache import DERR_CONTEXT, DERR_KV_PAGE, entry_slots

# pi to 60 digits
PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


def angle(position: int, inv_freq: float) -> float:
    """position * inv_freq reduced to (-pi, pi] in exact arithmetic."""
    x = Fraction(position) * Fraction(float(inv_freq)) / (2 * PI)
    x -= x.__floor__()
    if x > Fraction(1, 2):
        x -= 1
    return float(x * 2 * PI)


def norm_rope(x, weight, positions, inv_freq, eps, interleaved):
    """x [T, H, D]; returns z of the same shape, NaN-free rows of x for tokens
    with a negative position (left to the caller to mask)."""
    t, _, d = x.shape
    y = x / np.sqrt((x * x).sum(-1, keepdims=True) / d + eps)
    if weight is not None:
        y = y * weight
    z = y.copy()
    half = len(inv_freq)
    a = 2 * np.arange(half) if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    for i in range(t):
        if positions[i] < 0:
            continue
        th = np.array([angle(int(positions[i]), f) for f in inv_freq])
        c, s = np.cos(th), np.sin(th)
        z[i, :, a] = (y[i, :, a].T * c - y[i, :, b].T * s).T
        z[i, :, b] = (y[i, :, b].T * c + y[i, :, a].T * s).T
    return z


def attention(q, k, v, tables, starts, ctx, scale, window=0, sink=0, prefix_table=(), prefix_len=0,
              k_scale=None, v_scale=None):
    """q [rows, Hq, D]; k, v [P, S, Hk, D]; returns a dict: out, lse, and for the
    tests' bounds mag (the largest scale * sum |q k| a row meets), spread
    (sum_e p_e |V_e|), seen (entries a row sees), mine (rows of a request) and
    the error bits."""
    rows, hq, d = q.shape
    pages, size, hk, _ = k.shape
    g = hq // hk
    out, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -np.inf)
    mag, spread = np.zeros((rows, hq)), np.zeros((rows, hq, d))
    seen, mine = np.zeros(rows, dtype=np.int64), np.zeros(rows, dtype=bool)
    err = 0

    def there(table, e):
        nonlocal err
        page, slot = entry_slots(table, e, size, pages)
        if (page < 0).any():
            err |= DERR_KV_PAGE
        keep = page >= 0
        return e[keep], page[keep], slot[keep]

    pcap = len(prefix_table) * size
    if prefix_len > pcap:
        err |= DERR_CONTEXT
    for b in range(len(tables)):
        n, cap = int(starts[b + 1]) - int(starts[b]), tables.shape[1] * size
        if n == 0:
            continue
        if ctx[b] > cap:
            err |= DERR_CONTEXT
        length = max(int(ctx[b]), 0)
        _, ppage, pslot = there(np.asarray(prefix_table), np.arange(min(max(prefix_len, 0), pcap)))
        hi = length - n + np.arange(n) + 1
        e = np.arange(max(0, min(length, cap)))
        sees = e < hi[:, None]
        if window:
            sees &= (e >= hi[:, None] - window) | (e < sink)
        e = e[sees.any(0)]
        e, page, slot = there(tables[b], e)
        sees = np.concatenate([np.ones((n, len(ppage)), bool), sees[:, e]], 1)
        page, slot = np.concatenate([ppage, page]), np.concatenate([pslot, slot])
        r = slice(int(starts[b]), int(starts[b + 1]))
        mine[r] = True
        seen[r] = sees.sum(1)
        for h in range(hq):
            kk, vv = k[page, slot, h // g], v[page, slot, h // g]
            if k_scale is not None:
                kk = kk * float(k_scale[h // g])
            if v_scale is not None:
                vv = vv * float(v_scale[h // g])
            with np.errstate(invalid="ignore"):
                z = scale * (q[r, h] @ kk.T)
                m = scale * (np.abs(q[r, h]) @ np.abs(kk).T)
            z = np.where(sees, z, -np.inf)
            ok = sees.any(1)
            if not ok.any():
                continue
            top = np.where(ok, np.max(z, axis=1, initial=-np.inf), 0.0)
            p = np.exp(z - top[:, None])
            total = p.sum(1)
            p = p / np.where(ok, total, 1.0)[:, None]
            # an entry that a row does not see counts for nothing, whatever it holds
            for i in range(n):
                s = sees[i]
                out[r.start + i, h] = p[i, s] @ vv[s]
                spread[r.start + i, h] = p[i, s] @ np.abs(vv[s])
                mag[r.start + i, h] = m[i, s].max(initial=0.0)
            lse[r, h] = np.where(ok, top + np.log(np.where(ok, total, 1.0)), -np.inf)
    return {"out": out, "lse": lse, "mag": mag, "spread": spread, "seen": seen, "mine": mine,
            "err": err}
