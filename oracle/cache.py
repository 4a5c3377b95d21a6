"""Oracle of the paged K/V cache operators (include/qsa_cache.h): append,
dense attention with the weight each entry received, eviction.

Plain numpy in binary64 and Python integers, request by request and head by
head, from the header's definitions.  Shares nothing with the CUDA library.
Caches and queries come in as the values they hold (binary64, scales not yet
applied)."""
from __future__ import annotations

import numpy as np

DERR_REQUEST, DERR_KV_PAGE, DERR_CONTEXT = 1, 4, 32


def e4m3_magnitudes() -> np.ndarray:
    """The 127 finite magnitudes of E4M3, ascending: index = the code."""
    code = np.arange(127)
    exp, man = code >> 3, code & 7
    return np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp.astype(float) - 10))


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """x rounded to the nearest E4M3 value (ties to the even code), magnitudes
    above 448 to 448, NaN kept."""
    mags = e4m3_magnitudes()
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - mags[lo], mags[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    r = np.where(up, mags[hi], mags[lo])
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def entry_slots(table_row, entries, page_size, num_pages):
    """(page, slot) of each entry; page -1 where the table holds no valid one."""
    entries = np.asarray(entries, dtype=np.int64)
    col = entries // page_size
    inside = col < len(table_row)
    page = np.where(inside, np.asarray(table_row, dtype=np.int64)[np.where(inside, col, 0)]
                    if len(table_row) else -1, -1)
    return np.where((page >= 0) & (page < num_pages), page, -1), entries % page_size


def attention(q, k, v, tables, ctx, next_n, scale, window=0, k_scale=None, v_scale=None):
    """q [rows, Hq, D]; k, v [P, S, Hk, D]; returns a dict: out, lse, weights
    [requests, cols*S] (what each entry received), mag [rows, Hq] (the largest
    scale * sum |q k| a row meets), spread [rows, Hq, D] (sum_e p_e |V_e|) and
    the error bits."""
    rows, hq, d = q.shape
    pages, size, hk, _ = k.shape
    reqs, cols = tables.shape
    g = hq // hk
    out = np.zeros((rows, hq, d))
    lse = np.full((rows, hq), -np.inf)
    weights = np.zeros((reqs, cols * size))
    mag, spread = np.zeros((rows, hq)), np.zeros((rows, hq, d))
    err = 0
    for b in range(reqs):
        if ctx[b] > cols * size:
            err |= DERR_CONTEXT
        for j in range(next_n):
            hi = int(ctx[b]) - next_n + j + 1
            lo = max(0, hi - window) if window else 0
            e = np.arange(lo, min(hi, cols * size))
            if e.size == 0:
                continue
            page, slot = entry_slots(tables[b], e, size, pages)
            if (page < 0).any():
                err |= DERR_KV_PAGE
            e, page, slot = e[page >= 0], page[page >= 0], slot[page >= 0]
            if e.size == 0:
                continue
            for h in range(hq):
                kk, vv = k[page, slot, h // g], v[page, slot, h // g]
                if k_scale is not None:
                    kk = kk * float(k_scale[h // g])
                if v_scale is not None:
                    vv = vv * float(v_scale[h // g])
                r = b * next_n + j
                z = scale * (kk @ q[r, h])
                m = z.max()
                p = np.exp(z - m)
                total = p.sum()
                p = p / total
                out[r, h] = p @ vv
                lse[r, h] = m + np.log(total)
                weights[b, e] += p
                mag[r, h] = scale * (np.abs(kk) @ np.abs(q[r, h])).max()
                spread[r, h] = p @ np.abs(vv)
    return {"out": out, "lse": lse, "weights": weights, "mag": mag, "spread": spread, "err": err}


def evict(sums, positions, ctx, tables, page_size, num_pages, budget, sink, recent):
    """Returns (kept, new_lens, sums_out, positions_out, moves, err); moves is
    a list of (request, from entry, to entry)."""
    reqs, cols = tables.shape
    kept = np.full((reqs, budget), -1, dtype=np.int64)
    lens = np.zeros(reqs, dtype=np.int64)
    sums_out = np.zeros((reqs, budget), dtype=np.float32)
    pos_out = np.full((reqs, budget), -1, dtype=np.int64)
    moves, err = [], 0
    cap = min(cols * page_size, sums.shape[1], positions.shape[1])
    for b in range(reqs):
        if ctx[b] > cap:
            err |= DERR_CONTEXT
        n = max(0, min(int(ctx[b]), cap))
        lens[b] = min(n, budget)
        place = list(range(min(n, budget)))
        if n > budget:
            pos = [int(x) for x in positions[b, :n]]
            newest = max(pos)

            def rank(e):
                safe = pos[e] < sink or pos[e] > newest - recent
                w = float(sums[b, e])
                nan = w != w
                return (not safe, nan, 0.0 if safe or nan else -w, e)

            stay = set(sorted(range(n), key=rank)[:budget])
            movers = [e for e in range(budget, n) if e in stay]
            holes = [e for e in range(budget) if e not in stay]
            assert len(movers) == len(holes)
            for src, dst in zip(movers, holes):
                place[dst] = src
                moves.append((b, src, dst))
                pages, _ = entry_slots(tables[b], [src, dst], page_size, num_pages)
                if (pages < 0).any():
                    err |= DERR_KV_PAGE
        kept[b, :len(place)] = place
        sums_out[b, :len(place)] = sums[b, place]
        pos_out[b, :len(place)] = positions[b, place]
    return kept, lens, sums_out, pos_out, moves, err


def apply_moves(cache, moves, tables):
    """A copy of a cache [P, S, ...] with the moves' entries copied."""
    out = cache.copy()
    size = cache.shape[1]
    for b, src, dst in moves:
        (ps, pd), (ss, sd) = entry_slots(tables[b], [src, dst], size, cache.shape[0])
        if ps >= 0 and pd >= 0:
            out[pd, sd] = cache[ps, ss]
    return out


def append(k, v, k_cache, v_cache, tables, token_to_request, entries, entry_cols=None,
           positions=None, entry_positions=None, weight_sums=None):
    """Copies of (k_cache, v_cache, entry_positions, weight_sums) with the
    tokens written (k, v already in the cache's values), and the error bits."""
    kc, vc = k_cache.copy(), v_cache.copy()
    ep = None if entry_positions is None else entry_positions.copy()
    ws = None if weight_sums is None else weight_sums.copy()
    reqs, cols = tables.shape
    size = k_cache.shape[1]
    cap = cols * size if entry_cols is None else min(cols * size, entry_cols)
    err = 0
    for t, (r, e) in enumerate(zip(token_to_request.tolist(), entries.tolist())):
        if e < 0:
            continue
        if not 0 <= r < reqs:
            err |= DERR_REQUEST
            continue
        if e >= cap:
            err |= DERR_CONTEXT
            continue
        (page,), (slot,) = entry_slots(tables[r], [e], size, k_cache.shape[0])
        if page < 0:
            err |= DERR_KV_PAGE
            continue
        kc[page, slot], vc[page, slot] = k[t], v[t]
        if ep is not None:
            ep[r, e] = e if positions is None else positions[t]
        if ws is not None:
            ws[r, e] = 0
    return kc, vc, ep, ws, err
