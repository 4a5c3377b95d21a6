"""Pins of the paged-cache oracle (oracle/cache.py): closed forms, invariants
and hand-worked examples, no GPU."""
import numpy as np
import pytest
import torch

from oracle import cache as C


def _paged(rng, lens, size, hk, d, cols=None):
    cols = cols or -(-max(max(lens), 1) // size)
    pages = len(lens) * cols
    tables = rng.permutation(pages).reshape(len(lens), cols)
    k, v = rng.standard_normal((2, pages, size, hk, d))
    return k, v, tables


def test_e4m3_rounding_matches_torch_on_every_code_and_midpoint():
    mags = C.e4m3_magnitudes()
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mags, codes)
    mid = (mags[1:] + mags[:-1]) / 2
    x = np.concatenate([mags, mid, np.nextafter(mid, 1e9), np.nextafter(mid, 0)])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(C.to_e4m3(x.astype(np.float64)), want)
    assert np.array_equal(C.to_e4m3(np.array([449.0, 1e9, -np.inf, 464.0])), [448, 448, -448, 448])
    assert np.isnan(C.to_e4m3(np.array([np.nan])))[0]


def test_attention_of_equal_keys_is_the_mean_and_the_weights_sum_to_one():
    rng = np.random.default_rng(1)
    k, v, tables = _paged(rng, [37, 5, 0], 8, 2, 4)
    k[:] = k[0, 0, 0]
    q = rng.standard_normal((3, 4, 4))
    r = C.attention(q, k, v, tables, [37, 5, 0], 1, 0.5)
    for b, n in ((0, 37), (1, 5)):
        page, slot = C.entry_slots(tables[b], np.arange(n), 8, len(k))
        for h in range(4):
            assert np.allclose(r["out"][b, h], v[page, slot, h // 2].mean(0))
        assert np.allclose(r["weights"][b, :n], 4 / n) and not r["weights"][b, n:].any()
    assert not r["out"][2].any() and np.isneginf(r["lse"][2]).all()


def test_attention_joins_from_its_halves_by_lse():
    rng = np.random.default_rng(2)
    k, v, tables = _paged(rng, [64], 16, 1, 8)
    q = rng.standard_normal((1, 3, 8))
    whole = C.attention(q, k, v, tables, [64], 1, 0.3)
    a = C.attention(q, k, v, tables[:, :2], [32], 1, 0.3)
    b = C.attention(q, k, v, tables[:, 2:], [32], 1, 0.3)
    m = np.logaddexp(a["lse"], b["lse"])
    assert np.allclose(m, whole["lse"])
    joined = (np.exp(a["lse"] - m)[..., None] * a["out"] + np.exp(b["lse"] - m)[..., None] * b["out"])
    assert np.allclose(joined, whole["out"])


def test_draft_rows_are_rows_of_shorter_contexts_and_windows_cut_the_front():
    rng = np.random.default_rng(3)
    k, v, tables = _paged(rng, [20], 8, 1, 4)
    q = rng.standard_normal((3, 2, 4))
    r = C.attention(q, k, v, tables, [20], 3, 0.5, window=6)
    for j in range(3):
        n = 20 - 3 + j + 1
        page, slot = C.entry_slots(tables[0], np.arange(n - 6, n), 8, len(k))
        z = 0.5 * k[page, slot, 0] @ q[j, 1]
        p = np.exp(z) / np.exp(z).sum()
        assert np.allclose(r["out"][j, 1], p @ v[page, slot, 0])
    # tokens before the first one see nothing
    r = C.attention(q, k, v, tables, [1], 3, 0.5)
    assert np.isneginf(r["lse"][:2]).all() and np.isfinite(r["lse"][2]).all()


def test_attention_counts_absent_pages_as_holes():
    rng = np.random.default_rng(4)
    k, v, tables = _paged(rng, [24], 8, 1, 4)
    q = rng.standard_normal((1, 1, 4))
    holed = tables.copy()
    holed[0, 1] = -1
    r = C.attention(q, k, v, holed, [24], 1, 0.5)
    joined = C.attention(q, k, v, tables[:, [0, 2]], [16], 1, 0.5)
    assert np.allclose(r["out"], joined["out"]) and r["err"] == C.DERR_KV_PAGE
    r = C.attention(q, k, v, tables, [40], 1, 0.5)
    assert r["err"] == C.DERR_CONTEXT


def test_evict_worked_example():
    #        entry      0    1    2    3    4    5    6    7
    sums = np.array([[.1, .5, .2, .9, .0, .3, .4, .0]], dtype=np.float32)
    pos = np.array([[0, 1, 2, 3, 4, 5, 6, 7]])
    # sink 1 protects entry 0, recent 1 entry 7; then 3 (.9), 1 (.5); budget 4
    # stay 0 1 3 7: entry 7 goes to the hole at 2
    got = C.evict(sums, pos, [8], np.array([[0]]), 8, 1, 4, 1, 1)
    kept, lens, so, po, moves, err = got
    assert kept.tolist() == [[0, 1, 7, 3]] and lens.tolist() == [4] and err == 0
    assert moves == [(0, 7, 2)] and po.tolist() == [[0, 1, 7, 3]]
    assert so.tolist() == [[np.float32(.1), .5, 0, np.float32(.9)]]


def test_evict_ties_nan_zero_and_short_requests():
    sums = np.array([[1, 1, 1, 1], [np.nan, -np.inf, -0.0, 0.0], [5, 6, 7, 8]], dtype=np.float32)
    pos = np.tile(np.arange(4), (3, 1))
    tables = np.arange(3).reshape(3, 1)
    kept, lens, *_ = C.evict(sums, pos, [4, 4, 2], tables, 4, 3, 3, 0, 0)
    assert kept.tolist() == [[0, 1, 2], [3, 1, 2], [0, 1, -1]] and lens.tolist() == [3, 3, 2]


@pytest.mark.parametrize("seed", range(20))
def test_evict_invariants(seed):
    rng = np.random.default_rng(seed)
    n, budget = int(rng.integers(2, 60)), int(rng.integers(1, 50))
    sink = int(rng.integers(0, budget // 2 + 1))
    recent = int(rng.integers(0, budget - sink + 1))
    sums = rng.integers(0, 6, (1, n)).astype(np.float32)
    pos = rng.permutation(n)[None]
    kept, lens, so, po, moves, _ = C.evict(sums, pos, [n], np.zeros((1, 8), int), 8, 1, budget,
                                           sink, recent)
    m = min(n, budget)
    stay = kept[0, :m]
    assert lens[0] == m and len(set(stay.tolist())) == m
    gone = sorted(set(range(n)) - set(stay.tolist()))
    if gone:
        safe = (pos[0] < sink) | (pos[0] > n - 1 - recent)
        assert not safe[gone].any()
        rest = [e for e in stay if not safe[e]]
        if rest:
            assert min(sums[0, rest]) >= max(sums[0, gone])
    for i, e in enumerate(stay):
        assert e == i or (e >= budget and i in set(gone))
    assert sorted(e for e in stay if e >= budget) == [s for _, s, _ in moves]
    assert np.array_equal(so[0, :m], sums[0, stay]) and np.array_equal(po[0, :m], pos[0, stay])


def test_append_writes_exactly_the_tokens_slots():
    rng = np.random.default_rng(6)
    k, v, tables = _paged(rng, [16, 16], 8, 1, 2)
    nk, nv = rng.standard_normal((2, 5, 1, 2))
    req, ent = np.array([0, 1, 1, 7, 0]), np.array([3, 9, -1, 0, 16])
    ep, ws = np.full((2, 16), 9), np.full((2, 16), 2.0)
    kc, vc, ep2, ws2, err = C.append(nk, nv, k, v, tables, req, ent, positions=np.arange(5) + 100,
                                     entry_positions=ep, weight_sums=ws)
    assert err == C.DERR_REQUEST | C.DERR_CONTEXT
    changed = np.argwhere((kc != k).any((2, 3)))
    assert sorted(map(tuple, changed.tolist())) == sorted(
        [(tables[0, 0], 3), (tables[1, 1], 1)])
    assert np.array_equal(vc[tables[1, 1], 1], nv[1])
    assert ep2[0, 3] == 100 and ep2[1, 9] == 101 and (ep2 != ep).sum() == 2
    assert (ws2 == 0).sum() == 2
