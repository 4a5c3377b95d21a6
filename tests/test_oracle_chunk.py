"""Pins of oracle/chunk.py: norms with rotation and attention of ragged chunks,
from identities and brute force, and against the other oracle of the cache."""
import math

import numpy as np
import pytest

from oracle import cache as C
from oracle import chunk as K


def _rng(seed=0):
    return np.random.default_rng(seed)


def test_angle_is_the_products_remainder():
    assert K.angle(1, 1.0) == 1.0
    assert K.angle(3, 1.0) == 3.0
    assert abs(K.angle(4, 1.0) - (4 - 2 * math.pi)) < 1e-15
    assert abs(math.cos(K.angle(10 ** 6, 1.0)) - math.cos(1e6)) < 1e-12
    # far out, where a binary64 product no longer holds the angle: by doubling
    a, x = 1, K.angle(1, 0.37)
    for _ in range(35):
        a, x = 2 * a, 2 * x
        assert abs(math.remainder(x - K.angle(a, 0.37), 2 * math.pi)) < 1e-9
        x = K.angle(a, 0.37)


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_keeps_lengths_and_turns_by_differences(inter):
    r = _rng(1)
    d, half = 32, 8
    f = (1e4 ** (-np.arange(half) / half)).astype(np.float32)
    x = r.normal(size=(6, 3, d))
    z = K.norm_rope(x, None, [0, 5, 5, 70, 1000, -1], f, 0.0, inter)
    # every row's mean square is one, and pairs keep theirs
    assert np.allclose((z * z).mean(-1), 1.0)
    # position 0 and the elements behind the rotated ones: the norm alone
    y = x / np.sqrt((x * x).mean(-1, keepdims=True))
    assert np.allclose(z[0], y[0]) and np.allclose(z[:5, :, 16:], y[:5, :, 16:])
    assert np.allclose(z[5], y[5])
    # a product depends on the positions' difference alone
    q, k = r.normal(size=(1, 1, d)), r.normal(size=(1, 1, d))

    def dot(a, b):
        return float((K.norm_rope(q, None, [a], f, 0.0, inter) *
                      K.norm_rope(k, None, [b], f, 0.0, inter)).sum())
    assert abs(dot(3, 10) - dot(1003, 1010)) < 1e-9
    assert abs(dot(3, 10) - dot(3, 11)) > 1e-6
    # one pair worked by hand: a quarter turn takes (1, 0) to (0, 1)
    e = np.zeros((1, 1, d))
    a, b = (0, 1) if inter else (0, 8)
    e[0, 0, a] = 1.0
    g = np.zeros(half, np.float64)
    g[0] = math.pi / 2
    z = K.norm_rope(e, np.full(d, 2.0), [1], g, 0.0, inter)[0, 0]
    assert abs(z[a]) < 1e-12 and abs(z[b] - 2 * math.sqrt(d)) < 1e-12


def _case(r, lens, new, hq=4, hk=2, d=8, size=8):
    cols = max(1, -(-max(lens) // size))
    pages = len(lens) * cols + 3
    k, v = r.normal(size=(pages, size, hk, d)), r.normal(size=(pages, size, hk, d))
    tables = r.permutation(pages)[:len(lens) * cols].reshape(len(lens), cols)
    starts = np.concatenate([[0], np.cumsum(new)])
    return r.normal(size=(starts[-1], hq, d)), k, v, tables, starts


@pytest.mark.parametrize("window", [0, 1, 5, 100])
def test_uniform_chunks_are_the_cache_oracles_drafts(window):
    r = _rng(2)
    lens = [17, 3, 0, 40]
    q, k, v, tables, starts = _case(r, lens, [3] * 4)
    a = K.attention(q, k, v, tables, starts, lens, 0.3, window)
    b = C.attention(q, k, v, tables, lens, 3, 0.3, window)
    assert np.allclose(a["out"], b["out"]) and np.allclose(a["lse"], b["lse"])


def test_sinks_and_windows_by_brute_force():
    r = _rng(3)
    lens, new = [23, 9, 31], [5, 9, 1]
    q, k, v, tables, starts = _case(r, lens, new)
    got = K.attention(q, k, v, tables, starts, lens, 0.5, 6, 3)
    t = 0
    for b, (ctx, n) in enumerate(zip(lens, new)):
        for j in range(n):
            pos = ctx - n + j
            seen = [e for e in range(pos + 1) if pos - e < 6 or e < 3]
            assert got["seen"][t] == len(seen)
            for h in range(4):
                w = [math.exp(0.5 * float(k[tables[b][e // 8], e % 8, h // 2] @ q[t, h])) for e in seen]
                vs = [v[tables[b][e // 8], e % 8, h // 2] for e in seen]
                want = sum(x * y for x, y in zip(w, vs)) / sum(w)
                assert np.allclose(got["out"][t, h], want)
                assert abs(got["lse"][t, h] - math.log(sum(w))) < 1e-12
            t += 1


def test_prefix_is_a_longer_context():
    r = _rng(4)
    lens, new, size = [11, 2, 24], [2, 2, 7], 8
    q, k, v, tables, starts = _case(r, lens, new)
    prefix = np.array([5, 1])
    a = K.attention(q, k, v, tables, starts, lens, 0.4, prefix_table=prefix, prefix_len=16)
    joined = np.concatenate([np.tile(prefix, (3, 1)), tables], 1)
    b = K.attention(q, k, v, joined, starts, [n + 16 for n in lens], 0.4)
    assert np.allclose(a["out"], b["out"]) and np.allclose(a["lse"], b["lse"])
    none = K.attention(q, k, v, tables, starts, lens, 0.4, prefix_table=prefix, prefix_len=0)
    alone = K.attention(q, k, v, tables, starts, lens, 0.4)
    assert np.array_equal(none["out"], alone["out"])
    assert size * 2 == 16


def test_rows_that_see_nothing_bad_pages_and_padding():
    r = _rng(5)
    lens = [4, 0, -3, 30]
    q, k, v, tables, starts = _case(r, [4, 0, 0, 24], [4, 2, 1, 2])
    tables = tables[:, :3]
    tables[3, 1] = 999
    k[tables[0, 0], 4:] = np.nan
    v[tables[0, 0], 4:] = np.inf
    q2 = np.concatenate([np.zeros_like(q[:2]), q, np.zeros_like(q[:1])])
    got = K.attention(q2, k, v, tables, starts + 2, lens, 0.4)
    assert got["err"] == K.DERR_KV_PAGE | K.DERR_CONTEXT
    assert not got["mine"][:2].any() and got["mine"][2:11].all() and not got["mine"][11]
    assert np.isfinite(got["out"]).all()
    assert (got["out"][6:9] == 0).all() and np.isinf(got["lse"][6:9]).all()
    assert list(got["seen"][9:11]) == [16, 16]          # 24 entries held, 8 of them absent
