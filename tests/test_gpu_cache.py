"""GPU parity of the paged K/V cache operators (include/qsa_cache.h) against
oracle/cache.py, through the binding.

Tolerances (per element, from the arithmetic; u = 2^-24):
  logit   |dz| <= D * 2^-23 * scale * sum |q k|: a binary32 dot of D exact
          products, each of at most D additions off by one unit of the running
          sum of magnitudes (the tensor core truncates, so 2u, not u);
  weight  relative 2|dz| (numerator and denominator) + 2^-20 (the exponential,
          the rescalings, the joins) + c * 2^-23, c the additions on the longest
          chain of a sum: at most one per 16 entries, + 32;
  output  weight's error times sum_e p_e |V_e|, + the rounding of the weights
          that multiply V: 2^-22 (FP16) or 2^-16 (BF16) as a pair of values,
          half an eps as one value (more than 32 query rows on a K/V head, or
          an E4M3 cache), + half an eps of the output's type times the value,
          + half the smallest subnormal of FP16;
  lse     |dz| + the weight's sum terms + 2^-22 |lse|;
  sums    the weight's relative error times the weight, + 2^-22 of the sum.
Indices, lengths, moved bytes and appended values are compared exactly."""
import threading

import numpy as np
import pytest
import torch

import sparse_paged_attention_qsa_gb300 as qsa
from oracle import cache as C

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
HALF = {F16: 2.0 ** -11, BF16: 2.0 ** -8}      # half a step, relative to the value


def _f64(t):
    return None if t is None else t.float().double().cpu().numpy()


def _values(shape, dtype, gen, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def make_cache(pages, size, hk, d, dtype, layout, gen):
    if layout == "packed":
        kv = _values((pages, size, 2, hk, d), dtype, gen)
        return kv[:, :, 0], kv[:, :, 1]
    if layout == "heads":
        return tuple(_values((pages, hk, size, d), dtype, gen).transpose(1, 2) for _ in range(2))
    if layout == "wide":                       # rows of a larger tensor: gaps everywhere
        big = _values((2, pages, size + 3, hk + 1, d + 16), dtype, gen)
        return big[0, :, :size, :hk, :d], big[1, :, 1:size + 1, 1:, 16:]
    return tuple(_values((pages, size, hk, d), dtype, gen) for _ in range(2))


class Case:
    """A batch over its own shuffled pages.  lens: cached tokens a request."""

    def __init__(self, lens, hq, hk, d, size, dtype=F16, cache=None, layout="split", next_n=1,
                 window=0, seed=0, cols=None, spare=2):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        cpu = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        cols = cols or max(1, -(-max(lens) // size))
        pages = len(lens) * cols + spare
        self.k, self.v = make_cache(pages, size, hk, d, cache, layout, gen)
        self.tables = torch.randperm(pages, generator=cpu)[:len(lens) * cols].view(
            len(lens), cols).to(torch.int32).to(DEV)
        self.ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.q = _values((len(lens) * next_n, hq, d), dtype, gen)
        self.k_scale = self.v_scale = None
        if cache == E4M3:
            self.k_scale = 0.25 + torch.rand(hk, generator=gen, device=DEV)
            self.v_scale = 0.25 + torch.rand(hk, generator=gen, device=DEV)
        self.next_n, self.window, self.size, self.lens = next_n, window, size, lens
        self.scale = d ** -0.5

    def oracle(self):
        return C.attention(_f64(self.q), _f64(self.k), _f64(self.v), self.tables.cpu().numpy(),
                           self.ctx.tolist(), self.next_n, self.scale, self.window,
                           _f64(self.k_scale), _f64(self.v_scale))

    def run(self, **kw):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        lse = torch.empty(self.q.shape[:2], device=DEV)
        out = qsa.qsa_paged_attention(self.q, self.k, self.v, self.tables, self.ctx,
                                      next_n=self.next_n, window=self.window,
                                      k_scale=self.k_scale, v_scale=self.v_scale, lse=lse,
                                      error_word=err, **kw)
        return out, lse, err


def bounds(c, r, entries):
    d = c.q.shape[2]
    dz = d * 2.0 ** -23 * r["mag"]
    weight = 2 * dz + 2.0 ** -20 + (entries / 16 + 32) * 2.0 ** -23
    rows_on_head = c.q.shape[1] // c.k.shape[2] * c.next_n
    if c.k.dtype == E4M3:
        pair = 2.0 ** -11                      # V is FP16 there, whatever q is
    elif rows_on_head > 32:
        pair = HALF[c.q.dtype]
    else:
        pair = {F16: 2.0 ** -22, BF16: 2.0 ** -16}[c.q.dtype]
    out = (weight[..., None] + pair) * r["spread"] + HALF[c.q.dtype] * np.abs(r["out"]) + 2.0 ** -25
    fin = np.where(np.isfinite(r["lse"]), np.abs(r["lse"]), 0.0)
    return out, weight + 2.0 ** -22 * fin, weight.max(initial=0.0)


def check(c, sums=False, rows=None, expect=None):
    r = c.oracle()
    if sums:
        cols = c.tables.shape[1] * c.size
        base = torch.rand((len(c.lens), cols), device=DEV)
        got_sums = torch.full((len(c.lens), cols + 3), 7.0, device=DEV)[:, :cols]
        out, lse, err = c.run(weight_sums=base, weight_sums_out=got_sums)
    else:
        out, lse, err = c.run()
    torch.cuda.synchronize()
    tol, tol_lse, rel = bounds(c, r, max(max(c.lens), 1))
    rows = slice(None) if rows is None else rows
    diff = np.abs(_f64(out) - r["out"])[rows]
    assert (diff <= tol[rows]).all(), (diff.max(), np.argwhere(~(diff <= tol[rows]))[:4])
    got, want = lse.double().cpu().numpy()[rows], r["lse"][rows]
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fin = np.isfinite(want)
    assert (np.abs(got - want)[fin] <= tol_lse[rows][fin]).all(), np.abs(got - want)[fin].max()
    if expect is not None:
        assert int(err.item()) == expect == r["err"]
    else:
        assert int(err.item()) == r["err"]
    if sums:
        g, base = got_sums.double().cpu().numpy(), base.double().cpu().numpy()
        for b, n in enumerate(c.lens):
            n = min(max(n, 0), g.shape[1])
            want = base[b, :n] + r["weights"][b, :n]
            assert (np.abs(g[b, :n] - want) <= rel * r["weights"][b, :n] + 2.0 ** -22 * want).all()
            assert (g[b, n:] == 7.0).all()     # behind the last entry: as it was
    return out, lse


# --- attention --------------------------------------------------------------------


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_types_and_dims(d, dtype, cache):
    check(Case([1, 63, 64, 65, 700, 0], 6, 2, d, 32, dtype, cache, seed=d), sums=True)


@pytest.mark.parametrize("layout", ["split", "packed", "heads", "wide"])
@pytest.mark.parametrize("size", [8, 16, 64, 256, 512])
def test_attention_layouts_and_page_sizes(size, layout):
    check(Case([5, 1000, 513], 4, 2, 64, size, BF16, layout=layout, seed=size))
    check(Case([130, 77], 4, 2, 128, size, F16, E4M3, layout=layout, seed=size + 1))


@pytest.mark.parametrize("hq,hk,next_n", [(1, 1, 1), (3, 1, 1), (5, 5, 1), (12, 4, 3), (16, 1, 1),
                                          (17, 1, 1), (16, 2, 4), (34, 2, 2), (40, 1, 2),
                                          (64, 1, 1), (65, 1, 1), (16, 1, 8), (100, 1, 3)])
@pytest.mark.parametrize("d", [64, 256])
def test_attention_head_groups(hq, hk, next_n, d):
    check(Case([300, 17, 2], hq, hk, d, 16, F16, next_n=next_n, seed=hq), sums=True)
    check(Case([150, 1], hq, hk, d, 64, BF16, E4M3, next_n=next_n, seed=hq + 1))


@pytest.mark.parametrize("hq,hk,next_n", [(3, 1, 1), (17, 1, 1), (12, 4, 3), (16, 1, 8), (64, 1, 1),
                                          (20, 1, 4)])
@pytest.mark.parametrize("d,dtype,cache", [(64, F16, F16), (128, BF16, E4M3), (256, BF16, BF16)])
def test_attention_cut_requests(hq, hk, next_n, d, dtype, cache):
    # long enough that every request is cut between CTAs, in few and in many pieces
    check(Case([2600], hq, hk, d, 32, dtype, cache, next_n=next_n, seed=hq), sums=True)
    check(Case([2049, 3, 1500, 0, 2600], hq, hk, d, 64, dtype, cache, next_n=next_n, seed=hq + 1),
          sums=True)


@pytest.mark.parametrize("hq,hk,next_n", [(1, 1, 1), (3, 1, 1), (12, 4, 3), (16, 2, 2), (16, 1, 1)])
@pytest.mark.parametrize("d,dtype,cache,lens", [
    (64, F16, F16, [1100, 5, 0, 700]), (64, BF16, E4M3, [2300, 2, 2299]), (128, F16, F16, [1000]),
    (128, BF16, E4M3, [1200, 1, 64, 1199]), (256, BF16, BF16, [600, 0, 31]), (256, F16, E4M3, [1030])])
def test_attention_in_one_cluster(hq, hk, next_n, d, dtype, cache, lens):
    # short work whose requests are still cut: joined within one cluster of CTAs
    check(Case(lens, hq, hk, d, 16, dtype, cache, next_n=next_n, seed=hq + d), sums=True)
    check(Case(lens, hq, hk, d, 64, dtype, cache, next_n=next_n, window=520, seed=hq))


def test_attention_worked_size_of_the_packed_cache():
    check(Case([519], 3, 1, 256, 512, F16, layout="packed", seed=3))


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 5000])
@pytest.mark.parametrize("next_n", [1, 4])
def test_attention_windows(window, next_n):
    check(Case([1, 3, 64, 129, 1000, 0], 8, 2, 128, 32, F16, next_n=next_n, window=window,
               seed=window), sums=True)


@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 1, 2 ** 31, 2 ** 62, 2 ** 63 - 1])
def test_attention_windows_past_every_capacity(window):
    # contexts shorter than the draft too: rows of it see nothing
    check(Case([1, 2, 7, 700, 0], 4, 2, 64, 16, F16, next_n=8, window=window, seed=19), sums=True)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [64] * 40, list(range(0, 130, 7)),
                                  [4000, 1, 1, 1, 0, 3999], [20000]])
def test_attention_ragged_batches(lens):
    check(Case(lens, 4, 1, 128, 64, BF16, seed=len(lens)), sums=True)
    check(Case(lens, 4, 2, 64, 16, F16, next_n=2, seed=len(lens) + 1))


def test_attention_many_requests():
    lens = [(7 * i) % 90 for i in range(2500)]         # more than one launch's request table
    c = Case(lens, 2, 1, 64, 16, F16, seed=8)
    check(c, sums=True)


def test_attention_does_not_read_what_is_masked():
    # NaN and infinities in every slot no row may see, and in entries that only the later
    # rows of a draft see: the rows that do not see them stay as they are
    for d, cache in ((128, F16), (64, E4M3), (256, BF16)):
        dtype = F16 if cache == E4M3 else cache
        c = Case([70, 129, 5], 4, 2, d, 16, dtype, cache, next_n=3, window=40, seed=d, spare=4)
        bad = torch.tensor([float("nan")], device=DEV)
        seen = torch.zeros(c.k.shape[:2], dtype=torch.bool, device=DEV)
        for b, n in enumerate(c.lens):
            e = torch.arange(max(0, n - 2 - 40), n - 2, device=DEV)       # row 0's entries
            seen[c.tables[b, e // 16].long(), e % 16] = True
        clean = c.run()[0].clone()
        for t in (c.k, c.v):
            x = torch.where(seen[..., None, None], t.float(), bad)
            x[~seen] = bad if cache == E4M3 else torch.tensor(
                [float("nan"), float("inf"), -float("inf"), float("nan")],
                device=DEV).repeat(d // 4)
            t.copy_(x.to(cache))
        out, lse, _ = c.run()
        assert torch.isfinite(out[0::3]).all()
        r = c.oracle()
        tol = bounds(c, r, 129)[0]
        for b in range(3):
            assert (np.abs(_f64(out) - r["out"])[3 * b] <= tol[3 * b]).all()
            assert torch.equal(out[3 * b], clean[3 * b])


def test_attention_extreme_logits():
    # one entry far above the others, logits past the range of exp, equal keys
    c = Case([300, 64], 4, 1, 64, 16, F16, seed=5)
    c.k[c.tables[0, 3].long(), 5] *= 40
    check(c)
    c.q *= 30
    check(c)
    c.k[:] = c.k[0, 0, 0]
    check(c, sums=True)


def _fill(t, x):
    raw = torch.tensor(x).to(t.dtype)
    if t.dtype == E4M3:
        t.view(torch.uint8).fill_(int(raw.view(torch.uint8)))
    else:
        t.fill_(raw.item())


@pytest.mark.parametrize("hq,lens", [(4, [300, 0, 17]), (4, [1100, 5]), (4, [9000, 5]),
                                     (16, [2300, 5]), (17, [700, 33]), (64, [1500])])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (F16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("peak", [False, True])
def test_attention_logits_past_binary32s_integers(peak, sign, dtype, cache, hq, lens):
    """Finite logits of 2^24 to 2^28 in base 2, where binary32 no longer holds a logit
    less 15.  Every entry's key is the same, but for one with peak: the others' weights are then
    0.  q and K have at most 8 bits and equal elements, so that the products' sums are exact and
    the logits' error does not enter the weights; scale, its product and the lse's conversion
    round at most 7 times, below 2^-21 of the lse."""
    top = 448.0 if cache == E4M3 else None
    for a in (1216, 1792, 2944, 4032) if cache == F16 else (6656, 14336, 40960, 57344):
        c = Case(lens, hq, 1, 64, 16, dtype, cache, seed=hq)
        b = top or float(a)
        if c.k_scale is not None:
            c.k_scale.fill_(0.5)
        c.q.fill_(a)
        _fill(c.k, sign * b * (0.5 if peak and sign > 0 else 1))
        if peak:
            for i, n in enumerate(lens):
                _fill(c.k[int(c.tables[i, n // 3 // 16]), n // 3 % 16],
                      sign * b * (1 if sign > 0 else 0.5))
        r = c.oracle()
        out, lse, err = c.run()
        n = max(lens)
        weight = 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23
        pair = 2.0 ** -11 if cache == E4M3 else HALF[dtype] if hq > 32 else 2.0 ** -22
        tol = (weight + pair) * r["spread"] + HALF[dtype] * np.abs(r["out"]) + 2.0 ** -25
        assert torch.isfinite(out).all()
        assert (np.abs(_f64(out) - r["out"]) <= tol).all(), np.abs(_f64(out) - r["out"]).max()
        got, fin = lse.double().cpu().numpy(), np.isfinite(r["lse"])
        assert np.abs(r["lse"][fin]).max() > 0.69 * 2 ** 23
        assert np.array_equal(np.isneginf(got), np.isneginf(r["lse"]))
        assert (np.abs(got - r["lse"])[fin] <= weight + 2.0 ** -21 * np.abs(r["lse"][fin])).all()
        assert int(err.item()) == 0


# rows of a K/V head, cached tokens and page: walked whole, in one cluster, cut and joined
_MODES = [(4, [300, 0, 17]), (16, [1100, 5]), (4, [9000, 5]), (17, [1500, 33]), (64, [1500])]


@pytest.mark.parametrize("hq,lens", _MODES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_values_up_to_bf16s_range(d, hq, lens):
    """BF16 values of 1e35 in one entry and 1e30 in all the others, equal ones included:
    their sum is finite in binary32, so every result is."""
    c = Case(lens, hq, 1, d, 16, BF16, seed=hq + d)
    c.v.mul_(1e30)
    for i, n in enumerate(lens):
        _fill(c.v[int(c.tables[i, n // 2 // 16]), n // 2 % 16, :, : d // 2], 1e35)
    out, _ = check(c)
    _fill(c.v, 1e34)
    check(c)


@pytest.mark.parametrize("hq,lens", _MODES)
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3), (BF16, BF16)])
@pytest.mark.parametrize("sign", [1, -1])
def test_weight_sums_of_large_logits(sign, dtype, cache, hq, lens):
    """Equal keys give equal weights however large the logits are (up to 2^28 in base 2): the
    weights' error is that of the exponential and of the sum, not of the lse's own rounding.
    The weight is 2^((z - m) - log2 l): z - m exact, log2 l below 32 off by 2^-18 (one unit of
    its own, half of one of the difference's), which makes ln 2 * 2^-18 of the weight; the sum
    l and the exponential as in `bounds`; the sum over heads at most 64 more additions."""
    for a in (64.0, 1216.0, 4032.0):
        c = Case(lens, hq, 1, 64, 16, dtype, cache, seed=hq)
        if c.k_scale is not None:
            c.k_scale.fill_(1.0)
        _fill(c.q, a)
        _fill(c.k, sign * (448.0 if cache == E4M3 else a))
        cols = c.tables.shape[1] * 16
        base, added = torch.zeros((len(lens), cols), device=DEV), torch.zeros(
            (len(lens), cols), device=DEV)
        c.run(weight_sums=base, weight_sums_out=added)
        got = added.double().cpu().numpy()
        for i, n in enumerate(lens):
            rel = 2.0 ** -18 + 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23 + 64 * 2.0 ** -24
            if n:
                assert (np.abs(got[i, :n] * n / hq - 1) <= rel).all(), np.abs(got[i, :n] * n / hq - 1).max()
            assert not got[i, n:].any()


def test_attention_bad_pages_and_contexts():
    c = Case([200, 90, 64, 33], 4, 2, 128, 32, BF16, seed=6)
    c.tables[0, 2] = -1
    c.tables[1, 0] = c.k.shape[0]
    c.tables[2, :] = 2 ** 31 - 1                  # every page absent: an empty row
    check(c, sums=True, expect=C.DERR_KV_PAGE)
    c = Case([64, 40], 4, 2, 128, 32, F16, seed=7)
    c.ctx[0] = 1000                               # the table holds 64
    c.ctx[1] = -5
    r = c.oracle()
    out, lse, err = c.run()
    tol = bounds(c, r, 64)[0]
    assert (np.abs(_f64(out) - r["out"]) <= tol).all() and int(err.item()) == C.DERR_CONTEXT
    assert torch.isneginf(lse[1]).all() and not out[1].any()
    c.window = 10                                 # the window lies past the table
    out, lse, err = c.run()
    assert torch.isneginf(lse).all() and not out.any()


def test_attention_no_table_and_no_pages():
    c = Case([5, 0], 4, 2, 64, 16, F16, seed=9)
    none = torch.empty((2, 0), dtype=torch.int32, device=DEV)
    out = qsa.qsa_paged_attention(c.q, c.k, c.v, none, c.ctx)
    assert not out.any()
    out = qsa.qsa_paged_attention(c.q, c.k[:0], c.v[:0], c.tables, c.ctx)
    assert not out.any()
    empty = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    out = qsa.qsa_paged_attention(c.q[:0], c.k, c.v, empty, c.ctx[:0])
    assert out.shape == (0, 4, 64)


def test_attention_strided_queries_and_outputs():
    c = Case([100, 37], 4, 2, 64, 16, F16, next_n=2, seed=10)
    big = torch.zeros((4, 8, 80), dtype=F16, device=DEV)
    big[:, ::2, 8:72] = c.q
    plain = c.run()[0]
    c.q = big[:, ::2, 8:72]
    out = torch.zeros((4, 6, 128), dtype=F16, device=DEV)
    view = out[:, 1:5, 32:96]
    c.run(out=view)
    assert torch.equal(view, plain)
    out[:, 1:5, 32:96] = 0
    assert not out.any()


def test_attention_repeats_bit_for_bit_and_sums_grow_in_place():
    c = Case([5000, 300, 1, 2047], 8, 2, 128, 64, F16, seed=11)
    sums = torch.rand((4, c.tables.shape[1] * 64), device=DEV)
    once = torch.empty_like(sums).copy_(sums)
    outs = [c.run(weight_sums=sums, weight_sums_out=once)[0].clone() for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    place = sums.clone()
    c.run(weight_sums=place, weight_sums_out=place)
    assert torch.equal(place, once)
    c.run(weight_sums=place, weight_sums_out=place)
    assert (place[0, :5000].double().sum() - sums[0, :5000].double().sum() - 16).abs() < 1e-2


def test_attention_past_32_bit_offsets():
    # a cache of 2^32 bytes and more in K and in V: its last pages
    pages, size, hk, d = 66000, 128, 2, 128
    k = torch.zeros((pages, size, hk, d), dtype=F16, device=DEV)
    v = torch.zeros((pages, size, hk, d), dtype=F16, device=DEV)
    assert k.numel() > 2 ** 31
    c = Case([300], 4, hk, d, size, F16, seed=12)
    out, lse, _ = c.run()
    far = torch.arange(pages - 3, pages, device=DEV)
    k[far], v[far] = c.k[c.tables[0].long()], c.v[c.tables[0].long()]
    got = qsa.qsa_paged_attention(c.q, k, v, far.to(torch.int32)[None], c.ctx)
    assert torch.equal(got, out)
    nk = _values((1, hk, d), F16, torch.Generator(device=DEV).manual_seed(1))
    qsa.qsa_paged_append(nk, nk, k, v, far.to(torch.int32)[None],
                         torch.zeros(1, dtype=torch.int32, device=DEV),
                         torch.tensor([383], device=DEV))
    assert torch.equal(k[-1, 127], nk[0]) and torch.equal(v[-1, 127], nk[0])
    sums = torch.zeros((1, 384), device=DEV)
    sums[0, 383] = 1
    qsa.qsa_evict_entries(sums, torch.arange(384, device=DEV, dtype=torch.int32)[None],
                          torch.tensor([384], dtype=torch.int32, device=DEV), k, v,
                          far.to(torch.int32)[None], 383)
    assert torch.equal(k[-1, 126], nk[0])          # ties: entry 382 is the one that goes


def test_attention_other_streams_threads_and_graphs():
    c = Case([5000, 64, 1, 300], 8, 2, 128, 64, BF16, seed=13)
    sums = torch.rand((4, c.tables.shape[1] * 64), device=DEV)
    want_sums = torch.zeros_like(sums)
    want, want_lse, _ = c.run(weight_sums=sums, weight_sums_out=want_sums)
    torch.cuda.synchronize()
    # buffers made inside the call belong to the stream it was given
    side = torch.cuda.Stream()
    got = [c.run(stream=side)[0] for _ in range(4)]
    got += [c.run(stream=side.cuda_stream)[0] for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)
    found = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            o = c.run()[0]
            s.synchronize()
            found.append(torch.equal(o, want))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert found == [True] * 3
    # two graphs that share one workspace, replayed in turn on new inputs
    need = qsa.qsa_paged_attention_workspace_bytes(c.k, c.v, c.tables, num_heads=8,
                                                   with_weights=True)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    outs, lses, sums_out = [], [], torch.zeros_like(sums)
    graphs = []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(weight_sums=sums, weight_sums_out=sums_out, workspace=ws)
        side.synchronize()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                o, l, _ = c.run(weight_sums=sums, weight_sums_out=sums_out, workspace=ws)
            outs.append(o)
            lses.append(l)
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, l in zip(outs, lses):
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    assert torch.equal(sums_out, want_sums)
    c.ctx.copy_(torch.tensor([70, 1, 0, 4000], dtype=torch.int32))
    new = c.run()[0].clone()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], new)


def test_calls_in_a_row_see_what_was_written_before_them():
    # no host wait between steps that rewrite, in place, what the calls read (the kernels are
    # launched while their predecessor drains): every step as if it had run alone
    gen = torch.Generator(device=DEV).manual_seed(17)
    for lens, cols in (([2000, 70, 900], 64), ([30, 5, 20], 1), ([900, 3], 30)):
        c = Case(lens, 8, 2, 128, 32, F16, seed=18, cols=cols)
        n = len(lens)
        steps = 12
        qs = _values((steps, *c.q.shape), F16, gen)
        nks = _values((steps, n, 2, 128), F16, gen)
        ctxs = torch.stack([c.ctx - 5 * i if i % 3 else c.ctx for i in range(steps)]).clamp(min=1)
        t2r = torch.arange(n, dtype=torch.int32, device=DEV)
        sums = torch.zeros((n, cols * 32), device=DEV)
        pos = torch.arange(cols * 32, dtype=torch.int32, device=DEV).repeat(n, 1)
        k0, v0 = c.k.clone(), c.v.clone()

        def step(i, wait):
            c.q.copy_(qs[i])
            c.ctx.copy_(ctxs[i])
            if wait:
                torch.cuda.synchronize()
            qsa.qsa_paged_append(nks[i], nks[i], c.k, c.v, c.tables, t2r, c.ctx.long() - 1,
                                 weight_sums=sums, entry_positions=pos)
            if wait:
                torch.cuda.synchronize()
            out = qsa.qsa_paged_attention(c.q, c.k, c.v, c.tables, c.ctx, weight_sums=sums,
                                          weight_sums_out=sums)
            if wait:
                torch.cuda.synchronize()
            return [out, *qsa.qsa_evict_entries(sums, pos, c.ctx, c.k, c.v, c.tables, 16)]

        def run(wait):
            c.k.copy_(k0)
            c.v.copy_(v0)
            sums.zero_()
            return [[t.clone() for t in step(i, wait)] for i in range(steps)]

        alone = run(True)
        for got, want in zip(run(False), alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


_FIRST_IN_A_GRAPH = """
import torch
import sparse_paged_attention_qsa_gb300 as qsa
torch.manual_seed(0)
k, v = torch.randn((2, 80, 64, 2, 128), device="cuda").half()
tables = torch.randperm(80, device="cuda").to(torch.int32).view(2, 40)
ctx = torch.tensor([2500, 700], dtype=torch.int32, device="cuda")
q = torch.randn((2, 8, 128), device="cuda").half()
sums = torch.rand((2, 2560), device="cuda")
added = torch.zeros_like(sums)
pos = torch.arange(2560, dtype=torch.int32, device="cuda").repeat(2, 1)
t2r = torch.arange(2, dtype=torch.int32, device="cuda")
def step(k, v):
    qsa.qsa_paged_append(q[:, :2], q[:, 2:4], k, v, tables, t2r, ctx.long() - 1)
    out = qsa.qsa_paged_attention(q, k, v, tables, ctx, weight_sums=sums, weight_sums_out=added)
    return [out, added, *qsa.qsa_evict_entries(sums, pos, ctx, k, v, tables, 600, num_sink=2)]
kg, vg = k.clone(), v.clone()
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(s):
    with torch.cuda.graph(g, stream=s):
        got = step(kg, vg)
torch.cuda.synchronize()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = step(k, v)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert torch.equal(k, kg) and torch.equal(v, vg)
"""


def test_first_calls_inside_a_graph_capture():
    # a fresh process whose first calls (the kernels' one-time set-up) are captured
    import subprocess
    import sys
    root = __file__.rsplit("/tests/", 1)[0]
    r = subprocess.run([sys.executable, "-c", _FIRST_IN_A_GRAPH], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


class Thin(Case):
    """A case under a wide table: pages only where a request has tokens, the other
    columns hold ids that may not be looked at."""

    def __init__(self, lens, hq, hk, d, size, cols, dtype=F16, cache=None, **kw):
        used = [-(-n // size) for n in lens]
        total = sum(used)
        super().__init__([total * size], hq, hk, d, size, dtype, cache, cols=total, spare=1, **kw)
        tables = torch.full((len(lens), cols), 2 ** 31 - 1, dtype=torch.int32)
        ids, at = self.tables[0].cpu(), 0
        for b, n in enumerate(used):
            tables[b, :n] = ids[at:at + n]
            at += n
        self.tables, self.lens = tables.to(DEV), lens
        self.ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
        gen = torch.Generator(device=DEV).manual_seed(len(lens))
        self.q = _values((len(lens) * self.next_n, hq, d), dtype, gen)


@pytest.mark.parametrize("hq,hk,next_n", [(17, 1, 1), (32, 1, 1), (33, 1, 1), (64, 1, 1), (16, 2, 4),
                                          (40, 1, 2)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_many_rows_of_heads_of_128(hq, hk, next_n, dtype):
    check(Case([300, 17, 2], hq, hk, 128, 16, dtype, next_n=next_n, seed=hq), sums=True)
    check(Case([2049, 3, 700, 0], hq, hk, 128, 64, dtype, next_n=next_n, window=1500, seed=hq + 1),
          sums=True)


@pytest.mark.parametrize("hk,rows,lens", [(76, 17, [1100, 40]), (100, 17, [1100]), (160, 17, [1100, 3]),
                                          (40, 2, [1100, 9]), (320, 1, [90, 0, 33]), (1024, 2, [20])])
def test_attention_more_heads_than_a_wave_holds(hk, rows, lens):
    # two runs a head, one, more heads than CTAs; clusters past one wave; whole requests
    check(Case(lens, hk * rows, hk, 64, 16, F16, seed=hk), sums=True)


@pytest.mark.parametrize("size", [1024, 4096, 65536])
@pytest.mark.parametrize("d,dtype,cache", [(64, BF16, BF16), (128, F16, E4M3), (256, F16, F16)])
def test_attention_large_pages(d, dtype, cache, size):
    check(Thin([5, size, size + 77], 3, 1, d, size, 4, dtype, cache, seed=size), sums=True)


@pytest.mark.parametrize("rows", [2, 20])
def test_attention_many_requests_of_a_long_table(rows):
    # several launches of walk and join over one workspace; long requests at both sides of
    # each launch's end
    lens = [(7 * i) % 60 for i in range(1100)]
    for b in (3, 500, 511, 512, 513, 1023, 1024, 1099):
        lens[b] = 4000 + b
    check(Thin(lens, rows, 1, 64, 64, 90, F16, seed=9), sums=True)


# --- append ------------------------------------------------------------------------


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("hk,d,size,layout", [(1, 256, 512, "packed"), (8, 128, 16, "split"),
                                              (3, 64, 8, "heads"), (5, 64, 32, "wide")])
@pytest.mark.parametrize("T", [1, 7, 300])
def test_append(T, hk, d, size, layout, dtype, cache):
    gen = torch.Generator(device=DEV).manual_seed(T)
    cpu = torch.Generator().manual_seed(T)
    reqs, cols = 3, -(-2 * T // size)
    k, v = make_cache(reqs * cols + 1, size, hk, d, cache, layout, gen)
    tables = torch.randperm(reqs * cols + 1, generator=cpu)[:reqs * cols].view(reqs, cols)
    tables = tables.to(torch.int32).to(DEV)
    big = _values((T, hk + 1, 2 * d), dtype, gen, std=20.0)
    nk, nv = big[:, :hk, :d], big[:, 1:, d:]
    if T > 5:
        nk[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 6e4], device=DEV)
    req = torch.randint(reqs, (T,), generator=cpu).to(torch.int32)
    ent = torch.randperm(min(2 * T, cols * size), generator=cpu)[:T]      # distinct
    if T > 5:
        ent[3] = -1
    ks = vs = None
    if cache == E4M3:
        ks, vs = 0.05 + torch.rand((2, hk), generator=gen, device=DEV)
    pos = torch.arange(T) + 2 ** 20
    ep = torch.full((reqs, cols * size), -7, dtype=torch.int32, device=DEV)
    sums = torch.ones((reqs, cols * size + 5), device=DEV)[:, 2:-3]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def stored(x, s):
        x = x.float().cpu().numpy()
        if cache != E4M3:
            return x.astype(np.float64)
        inverse = np.float32(1) / s.cpu().numpy()[:, None]        # both steps in binary32
        return C.to_e4m3((x * inverse).astype(np.float64))

    want = C.append(stored(nk, ks), stored(nv, vs), _f64(k), _f64(v), tables.cpu().numpy(),
                    req.numpy(), ent.numpy(), None, pos.numpy(), ep.cpu().numpy(),
                    sums.cpu().numpy())
    qsa.qsa_paged_append(nk, nv, k, v, tables, req.to(DEV), ent.to(DEV), k_scale=ks, v_scale=vs,
                         positions=pos.to(DEV), entry_positions=ep, weight_sums=sums,
                         error_word=err)
    for got, exp in zip((k, v), want):
        assert np.array_equal(_f64(got), exp, equal_nan=True)
    assert np.array_equal(ep.cpu().numpy(), want[2]) and np.array_equal(sums.cpu().numpy(), want[3])
    assert int(err.item()) == want[4] == 0


def test_append_bad_tokens_and_defaults():
    gen = torch.Generator(device=DEV).manual_seed(2)
    k, v = make_cache(6, 8, 2, 64, F16, "split", gen)
    tables = torch.tensor([[0, 1, 9], [3, -1, 5]], dtype=torch.int32, device=DEV)
    before = k.clone()
    nk = _values((8, 2, 64), F16, gen)
    req = torch.tensor([0, 1, 1, 2, -1, 0, 1, 0], dtype=torch.int32)
    ent = torch.tensor([17, 8, 16, 0, 0, 24, 1 << 40, -(1 << 40)])
    ep = torch.full((2, 24), -7, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = C.append(_f64(nk), _f64(nk), _f64(k), _f64(v), tables.cpu().numpy(), req.numpy(),
                    ent.numpy(), 24, None, ep.cpu().numpy())
    qsa.qsa_paged_append(nk, nk, k, v, tables, req.to(DEV), ent.to(DEV), entry_positions=ep,
                         error_word=err)
    assert np.array_equal(_f64(k), want[0]) and np.array_equal(_f64(v), want[1])
    assert np.array_equal(ep.cpu().numpy(), want[2])
    assert int(err.item()) == want[4] == 1 | 4 | 32
    assert (k != before).any(dim=(2, 3)).sum() == 1
    # per-entry arrays shorter than the table bound the entries too
    err.zero_()
    qsa.qsa_paged_append(nk[:1], nk[:1], k, v, tables, req[:1].to(DEV), ent[:1].to(DEV),
                         entry_positions=ep[:, :17], error_word=err)
    assert int(err.item()) == 32
    qsa.qsa_paged_append(nk[:0], nk[:0], k, v, tables, req[:0].to(DEV), ent[:0].to(DEV))


def test_append_takes_the_metadata_builders_outputs():
    gen = torch.Generator(device=DEV).manual_seed(3)
    k, v = make_cache(8, 16, 2, 64, BF16, "split", gen)
    tables = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    qsl = torch.tensor([0, 3, 10], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 40], dtype=torch.int32, device=DEV)
    common = torch.zeros(12, dtype=torch.int64, device=DEV)
    md = qsa.qsa_build_metadata(qsl, lens, tables, 12, storage_block_size=16, compress_ratio=1,
                                common_slot_mapping=common, num_mapped_tokens=10)
    nk = _values((12, 2, 64), BF16, gen)
    before = k.clone()
    qsa.qsa_paged_append(nk, nk, k, v, tables, md["token_to_req"], md["logical_positions"])
    flat = k.view(8 * 16, 2, 64)
    assert torch.equal(flat[:3], nk[:3]) and torch.equal(flat[64 + 33:64 + 40], nk[3:10])
    assert (k != before).any(dim=(2, 3)).sum() == 10


# --- eviction -----------------------------------------------------------------------


def _evict_case(lens, budget, sink, recent, size=16, hk=2, d=64, dtype=F16, layout="split", seed=0,
                kind="spread", cols=None):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    cols = cols or max(1, -(-max(max(lens), budget) // size))
    k, v = make_cache(len(lens) * cols + 1, size, hk, d, dtype, layout, gen)
    tables = torch.randperm(len(lens) * cols + 1, generator=cpu)[:len(lens) * cols]
    tables = tables.view(len(lens), cols).to(torch.int32).to(DEV)
    W = cols * size
    if kind == "spread":
        sums = torch.rand((len(lens), W), generator=cpu).pow(6)
    elif kind == "ties":
        sums = torch.randint(0, 3, (len(lens), W), generator=cpu).float()
    else:
        pick = torch.tensor([0.0, -0.0, 1.0, -1.0, float("inf"), -float("inf"), float("nan"), 1e-45,
                             3e38, 1.0000001])
        sums = pick[torch.randint(0, 10, (len(lens), W), generator=cpu)]
    pos = torch.stack([torch.randperm(W, generator=cpu) for _ in lens]).to(torch.int32)
    return k, v, tables, sums.to(DEV), pos.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def _check_evict(case, budget, sink, recent, expect=0):
    k, v, tables, sums, pos, ctx = case
    want = C.evict(sums.cpu().numpy(), pos.cpu().numpy(), ctx.tolist(), tables.cpu().numpy(),
                   k.shape[1], k.shape[0], budget, sink, recent)
    wk, wv = (C.apply_moves(_f64(t), want[4], tables.cpu().numpy()) for t in (k, v))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = qsa.qsa_evict_entries(sums, pos, ctx, k, v, tables, budget, num_sink=sink,
                                num_recent=recent, error_word=err)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w, equal_nan=g.is_floating_point())
    assert np.array_equal(_f64(k), wk) and np.array_equal(_f64(v), wv)
    assert int(err.item()) == want[5] == expect
    return got


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([1, 2, 0, 5], 1, 0, 0), ([17], 16, 4, 4), ([2064] * 3, 2048, 4, 256), ([100, 300, 50], 64, 0, 64),
    ([100, 300, 50], 64, 64, 0), ([33, 64, 65], 64, 2, 8), ([1000, 4097], 999, 0, 1),
    ([9000, 20, 3000], 2500, 4, 128), ([5000], 4999, 0, 0), ([3], 40, 1, 1)])
def test_evict(lens, budget, sink, recent, kind):
    _check_evict(_evict_case(lens, budget, sink, recent, seed=len(lens) + budget, kind=kind),
                 budget, sink, recent)


@pytest.mark.parametrize("n", [70000, 140000])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict_long_requests(n, kind):
    _check_evict(_evict_case([n, n // 3], 9000, 4, 500, size=512, hk=1, seed=n, kind=kind), 9000, 4,
                 500)


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("budget", [1, 5, 16, 40])
def test_evict_short_requests_of_a_long_table(budget, kind):
    # a cluster's slices of a few entries, some of none
    lens = [1, 2, 9, 10, 11, 17, 31, 33, 80]
    _check_evict(_evict_case(lens, budget, budget // 4, budget // 4, seed=budget, kind=kind,
                             cols=2100), budget, budget // 4, budget // 4)


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("reqs,cap,budget", [(2, 200704, 9000), (19, 200704, 700), (21, 100352, 20000),
                                             (40, 50176, 5000), (78, 25088, 24000), (200, 25088, 64)])
def test_evict_keys_outside_shared_memory(reqs, cap, budget, kind):
    """Tables whose slices pass what a CTA's shared memory holds: clusters of 8, 4, 2 and 1.
    A few long requests, one of them the whole table."""
    gen = torch.Generator(device=DEV).manual_seed(reqs)
    cpu = torch.Generator().manual_seed(reqs)
    size = 512
    lens = [(37 * b) % 100 for b in range(reqs)]
    lens[0], lens[reqs // 2], lens[-1] = cap, budget + 1, cap - 12345
    used = [-(-n // size) for n in lens]
    k, v = make_cache(sum(used) + 1, size, 1, 64, F16, "split", gen)
    ids, at = torch.randperm(sum(used) + 1, generator=cpu), 0
    tables = torch.full((reqs, cap // size), -1, dtype=torch.int32)
    for b, n in enumerate(used):
        tables[b, :n] = ids[at:at + n]
        at += n
    if kind == "spread":
        sums = torch.rand((reqs, cap), generator=cpu).pow(6)
    elif kind == "ties":
        sums = torch.randint(0, 3, (reqs, cap), generator=cpu).float()
    else:
        pick = torch.tensor([0.0, -0.0, 1.0, -1.0, float("inf"), -float("inf"), float("nan"), 1e-45,
                             3e38, 1.0000001])
        sums = pick[torch.randint(0, 10, (reqs, cap), generator=cpu)]
    pos = torch.randperm(cap, generator=cpu).to(torch.int32).repeat(reqs, 1)
    case = (k, v, tables.to(DEV), sums.to(DEV), pos.to(DEV),
            torch.tensor(lens, dtype=torch.int32, device=DEV))
    _check_evict(case, budget, 4, min(500, budget // 2))


@pytest.mark.parametrize("size", [1024, 65536])
def test_append_and_evict_large_pages(size):
    lens, budget = [size + 40, 70, size], size - 5
    k, v, tables, sums, pos, ctx = case = _evict_case(lens, budget, 2, 9, size, 1, 64, BF16, seed=size)
    _check_evict(case, budget, 2, 9)
    nk = _values((3, 1, 64), BF16, torch.Generator(device=DEV).manual_seed(1))
    t2r = torch.arange(3, dtype=torch.int32, device=DEV)
    ent = torch.tensor([size - 1, size, 2 * size - 1], device=DEV)
    qsa.qsa_paged_append(nk, nk, k, v, tables, t2r, ent)
    for i, e in enumerate(ent.tolist()):
        assert torch.equal(k[int(tables[i, e // size]), e % size], nk[i])


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("layout,hk,d,size", [("packed", 1, 256, 512), ("heads", 3, 64, 8),
                                              ("wide", 5, 128, 32)])
def test_evict_moves_every_layout(layout, hk, d, size, dtype):
    _check_evict(_evict_case([700, 90], 80, 3, 11, size, hk, d, dtype, layout, seed=d), 80, 3, 11)


def test_evict_bad_pages_contexts_and_positions():
    case = _evict_case([300, 200], 100, 0, 0, seed=21)
    case[2][0, 1] = -1
    case[2][1, 9] = 2 ** 30
    _check_evict(case, 100, 0, 0, expect=C.DERR_KV_PAGE)
    case = _evict_case([64, 64], 20, 2, 2, seed=22)
    case[5][0], case[5][1] = 1 << 20, -3
    _check_evict(case, 20, 2, 2, expect=C.DERR_CONTEXT)
    # equal positions may protect more than the budget: the first stay; far positions do not wrap
    case = _evict_case([64, 64, 64], 20, 2, 2, seed=23)
    case[4][0] = 0
    case[4][1] = -2 ** 31
    case[4][2, 5] = 2 ** 31 - 1
    _check_evict(case, 20, 2, 2)


@pytest.mark.parametrize("lens,budget", [([900, 1300, 20], 256), ([40000, 100], 3000)])
def test_evict_into_wider_arrays(lens, budget):
    case = _evict_case(lens, budget, 4, 32, seed=25)
    k, v, tables, sums, pos, ctx = case
    kk, vv = k.clone(), v.clone()
    plain = _check_evict(case, budget, 4, 32)
    so = torch.full((len(lens), sums.shape[1] + 3), 7.0, device=DEV)
    po = torch.full((len(lens), sums.shape[1]), -9, dtype=torch.int32, device=DEV)
    got = qsa.qsa_evict_entries(sums, pos, ctx, kk, vv, tables, budget, num_sink=4, num_recent=32,
                                weight_sums_out=so[:, 1:], entry_positions_out=po)
    assert got[2].data_ptr() == so[:, 1:].data_ptr() and got[3] is po
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    assert torch.equal(so[:, 1:budget + 1], plain[2]) and torch.equal(po[:, :budget], plain[3])
    assert (so[:, 0] == 7).all() and (so[:, budget + 1:] == 7).all() and (po[:, budget:] == -9).all()
    assert torch.equal(k, kk) and torch.equal(v, vv)


def test_evict_strided_inputs_repeats_and_graph():
    lens, budget = [900, 1300], 256
    case = _evict_case(lens, budget, 4, 32, seed=24)
    k, v, tables, sums, pos, ctx = case
    wide = torch.zeros((2, sums.shape[1] + 9), device=DEV)
    wide[:, 4:-5] = sums
    kk, vv = k.clone(), v.clone()
    plain = _check_evict(case, budget, 4, 32)
    again = qsa.qsa_evict_entries(wide[:, 4:-5], pos, ctx, kk, vv, tables, budget, num_sink=4,
                                  num_recent=32)
    assert all(torch.equal(a, b) for a, b in zip(plain, again))
    assert torch.equal(k, kk) and torch.equal(v, vv)
    # the same call again moves the same entries: sources are never written
    again = qsa.qsa_evict_entries(sums, pos, ctx, kk, vv, tables, budget, num_sink=4, num_recent=32)
    assert all(torch.equal(a, b) for a, b in zip(plain, again)) and torch.equal(k, kk)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = qsa.qsa_evict_entries(sums, pos, ctx, kk, vv, tables, budget, num_sink=4,
                                        num_recent=32)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plain, got))


# --- together -------------------------------------------------------------------------


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
def test_bounded_cache_decode(dtype, cache):
    """Steps of a decode loop on a bounded cache: append the new token, attend over what is
    cached while adding up the weights, evict when a request reaches its limit.  Every step
    against the oracle on the state the step started from."""
    hq, hk, d, size, budget, limit, steps = 8, 2, 64, 16, 40, 48, 30
    gen = torch.Generator(device=DEV).manual_seed(31)
    lens = [45, 3, 47]
    reqs, cols = len(lens), limit // size
    k, v = make_cache(reqs * cols, size, hk, d, cache, "split", gen)
    tables = torch.randperm(reqs * cols, generator=torch.Generator().manual_seed(1)).view(
        reqs, cols).to(torch.int32).to(DEV)
    ks = vs = None
    if cache == E4M3:
        ks, vs = torch.full((2, hk), 0.02, device=DEV)
    pos = torch.arange(limit, dtype=torch.int32, device=DEV).repeat(reqs, 1)
    sums = torch.rand((reqs, limit), generator=gen, device=DEV)
    seen = torch.tensor(lens, device=DEV)                  # tokens so far: the next position
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    evictions = 0
    for step in range(steps):
        nk, nv = _values((2, reqs, hk, d), dtype, gen)
        t2r = torch.arange(reqs, dtype=torch.int32, device=DEV)
        entries = ctx.long()

        def stored(x, s):
            x = x.float().cpu().numpy()
            if s is None:
                return x.astype(np.float64)
            inverse = np.float32(1) / s.cpu().numpy()[:, None]
            return C.to_e4m3((x * inverse).astype(np.float64))

        want = C.append(stored(nk, ks), stored(nv, vs), _f64(k), _f64(v), tables.cpu().numpy(),
                        t2r.cpu().numpy(), entries.cpu().numpy(), limit, seen.cpu().numpy(),
                        pos.cpu().numpy(), sums.cpu().numpy())
        qsa.qsa_paged_append(nk, nv, k, v, tables, t2r, entries, k_scale=ks, v_scale=vs,
                             positions=seen, entry_positions=pos, weight_sums=sums)
        assert np.array_equal(_f64(k), want[0]) and np.array_equal(_f64(v), want[1])
        assert np.array_equal(pos.cpu().numpy(), want[2])
        assert np.array_equal(sums.cpu().numpy(), want[3])
        ctx, seen = ctx + 1, seen + 1
        q = _values((reqs, hq, d), dtype, gen)
        r = C.attention(_f64(q), _f64(k), _f64(v), tables.cpu().numpy(), ctx.tolist(), 1, d ** -0.5,
                        0, _f64(ks), _f64(vs))
        old = sums.double().cpu().numpy()
        out = qsa.qsa_paged_attention(q, k, v, tables, ctx, k_scale=ks, v_scale=vs,
                                      weight_sums=sums, weight_sums_out=sums)
        c = Case.__new__(Case)
        c.q, c.k, c.next_n = q, k, 1
        tol, _, rel = bounds(c, r, limit)
        assert (np.abs(_f64(out) - r["out"]) <= tol).all()
        want = old + r["weights"]
        assert (np.abs(sums.double().cpu().numpy() - want)
                <= rel * r["weights"] + 2.0 ** -22 * want).all()
        if int(ctx.max()) == limit:
            evictions += 1
            w = C.evict(sums.cpu().numpy(), pos.cpu().numpy(), ctx.tolist(), tables.cpu().numpy(),
                        size, k.shape[0], budget, 2, 8)
            wk = C.apply_moves(_f64(k), w[4], tables.cpu().numpy())
            kept, ctx, s2, p2 = qsa.qsa_evict_entries(sums, pos, ctx, k, v, tables, budget,
                                                      num_sink=2, num_recent=8)
            for g, e in zip((kept, ctx, s2, p2), w):
                assert np.array_equal(g.cpu().numpy(), e)
            assert np.array_equal(_f64(k), wk)
            sums, pos = torch.zeros_like(sums), torch.full_like(pos, -1)
            sums[:, :budget], pos[:, :budget] = s2, p2
            newest = (seen - 1).to(torch.int32)
            for b in range(reqs):
                held = set(pos[b, :int(ctx[b])].tolist())
                top = int(newest[b])
                assert {0, 1} <= held and set(range(max(0, top - 7), top + 1)) <= held
    assert evictions >= 3


@pytest.mark.parametrize("each", [True, False])
@pytest.mark.parametrize("dtype,cache,n", [(F16, F16, 1), (BF16, E4M3, 3), (BF16, BF16, 8)])
def test_bounded_cache_decode_with_arrays_in_turn(dtype, cache, n, each):
    """The loop that the README shows: the eviction writes the per-entry arrays that the next
    step reads, nothing is copied between steps.  n new tokens a request and step; an eviction
    each step, or when a request has no room for the next one."""
    hq, hk, d, size, budget, cols, steps = 8, 2, 64, 16, 40, 4, 37 if n == 1 else 14
    gen = torch.Generator(device=DEV).manual_seed(33)
    lens0 = [45, 0, 52]
    reqs, limit = len(lens0), cols * size
    k_cache, v_cache = make_cache(reqs * cols, size, hk, d, cache, "split", gen)
    tables = torch.randperm(reqs * cols, generator=torch.Generator().manual_seed(2)).view(
        reqs, cols).to(torch.int32).to(DEV)
    ks = vs = None
    if cache == E4M3:
        ks, vs = torch.full((2, hk), 0.02, device=DEV)
    entry_positions = torch.arange(limit, dtype=torch.int32, device=DEV).repeat(reqs, 1)
    sums = torch.rand((reqs, limit), generator=gen, device=DEV)
    sums2, entry_positions2 = torch.empty_like(sums), torch.empty_like(entry_positions)
    seen = torch.tensor(lens0, device=DEV)
    lens = seen.to(torch.int32)
    t2r = torch.arange(reqs, dtype=torch.int32, device=DEV).repeat_interleave(n)
    j = torch.arange(n, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    evictions = 0
    for step in range(steps):
        k_new, v_new = _values((2, reqs * n, hk, d), dtype, gen)
        entries = (lens.long()[:, None] + j).flatten()
        positions = (seen[:, None] + j).flatten()
        lens, seen = lens + n, seen + n
        qsa.qsa_paged_append(k_new, v_new, k_cache, v_cache, tables, t2r, entries, k_scale=ks,
                             v_scale=vs, positions=positions, entry_positions=entry_positions,
                             weight_sums=sums, error_word=err)
        for b in range(reqs):                  # the new tokens are there, and weigh nothing yet
            at = slice(int(lens[b]) - n, int(lens[b]))
            assert entry_positions[b, at].tolist() == positions.view(reqs, n)[b].tolist()
            assert not sums[b, at].any()
        q = _values((reqs * n, hq, d), dtype, gen)
        old = sums.double().cpu().numpy()
        r = C.attention(_f64(q), _f64(k_cache), _f64(v_cache), tables.cpu().numpy(), lens.tolist(),
                        n, d ** -0.5, 0, _f64(ks), _f64(vs))
        out = qsa.qsa_paged_attention(q, k_cache, v_cache, tables, lens, next_n=n, k_scale=ks,
                                      v_scale=vs, weight_sums=sums, weight_sums_out=sums,
                                      error_word=err)
        c = Case.__new__(Case)
        c.q, c.k, c.next_n = q, k_cache, n
        tol, _, rel = bounds(c, r, limit)
        assert (np.abs(_f64(out) - r["out"]) <= tol).all()
        got = sums.double().cpu().numpy()
        for b, m in enumerate(lens.tolist()):
            want = old[b, :m] + r["weights"][b, :m]
            assert (np.abs(got[b, :m] - want)
                    <= rel * r["weights"][b, :m] + 2.0 ** -22 * want).all()
        if not each and int(lens.max()) + n <= limit:
            continue
        evictions += int(lens.max()) > budget
        w = C.evict(sums.cpu().numpy(), entry_positions.cpu().numpy(), lens.tolist(),
                    tables.cpu().numpy(), size, k_cache.shape[0], budget, 2, 8)
        wk, wv = (C.apply_moves(_f64(t), w[4], tables.cpu().numpy()) for t in (k_cache, v_cache))
        kept, lens, _, _ = qsa.qsa_evict_entries(
            sums, entry_positions, lens, k_cache, v_cache, tables, budget, num_sink=2, num_recent=8,
            weight_sums_out=sums2, entry_positions_out=entry_positions2, error_word=err)
        sums, sums2 = sums2, sums
        entry_positions, entry_positions2 = entry_positions2, entry_positions
        for g, e in zip((kept, lens, sums[:, :budget], entry_positions[:, :budget]), w):
            assert np.array_equal(g.cpu().numpy(), e)
        assert np.array_equal(_f64(k_cache), wk) and np.array_equal(_f64(v_cache), wv)
    assert evictions >= 2 and int(err.item()) == 0


def test_bounded_cache_decode_in_two_graphs():
    """The README's loop captured: one graph for each direction of the per-entry arrays and of the
    lengths, replayed in turn, against the same steps run one by one."""
    hq, hk, d, size, budget, cols, steps = 8, 2, 128, 16, 300, 24, 7
    lens0 = [300, 12, 331]
    reqs, limit = len(lens0), cols * size
    gen = torch.Generator(device=DEV).manual_seed(41)
    k0, v0 = make_cache(reqs * cols, size, hk, d, F16, "split", gen)
    tables = torch.randperm(reqs * cols, generator=torch.Generator().manual_seed(3)).view(
        reqs, cols).to(torch.int32).to(DEV)
    t2r = torch.arange(reqs, dtype=torch.int32, device=DEV)
    new = _values((steps, 2, reqs, hk, d), F16, gen)
    qs = _values((steps, reqs, hq, d), F16, gen)
    sums0 = torch.rand((reqs, limit), generator=gen, device=DEV)

    class State:
        def __init__(self):
            self.k, self.v = k0.clone(), v0.clone()
            self.seen = torch.tensor(lens0, device=DEV)
            self.lens = [self.seen.to(torch.int32), torch.zeros(reqs, dtype=torch.int32, device=DEV)]
            self.sums = [sums0.clone(), torch.full_like(sums0, 9.0)]
            self.pos = [torch.arange(limit, dtype=torch.int32, device=DEV).repeat(reqs, 1),
                        torch.full((reqs, limit), -5, dtype=torch.int32, device=DEV)]
            self.new, self.q = new[0].clone(), qs[0].clone()

        def step(self, way):
            lens, sums, pos = self.lens[way], self.sums[way], self.pos[way]
            entries = lens.long()
            lens += 1
            qsa.qsa_paged_append(self.new[0], self.new[1], self.k, self.v, tables, t2r, entries,
                                 positions=self.seen, entry_positions=pos, weight_sums=sums)
            self.seen += 1
            out = qsa.qsa_paged_attention(self.q, self.k, self.v, tables, lens, weight_sums=sums,
                                          weight_sums_out=sums)
            kept = qsa.qsa_evict_entries(
                sums, pos, lens, self.k, self.v, tables, budget, num_sink=2, num_recent=8,
                new_lens=self.lens[1 - way], weight_sums_out=self.sums[1 - way],
                entry_positions_out=self.pos[1 - way])[0]
            return out, kept

        def feed(self, i):
            self.new.copy_(new[i])
            self.q.copy_(qs[i])

        def all(self):
            return [self.k, self.v, self.seen, *self.lens, *self.sums, *self.pos]

    eager, want = State(), []
    for i in range(steps):
        eager.feed(i)
        want.append([t.clone() for t in eager.step(i % 2)])
    torch.cuda.synchronize()
    s, graphs, results = State(), [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for way in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                results.append(s.step(way))
            graphs.append(g)
    torch.cuda.synchronize()
    for i in range(steps):                      # nothing waits between the replays
        s.feed(i)
        graphs[i % 2].replay()
        want_out, want_kept = want[i]
        out, kept = results[i % 2]
        assert torch.equal(out, want_out) and torch.equal(kept, want_kept)
    assert all(torch.equal(a, b) for a, b in zip(s.all(), eager.all()))
    assert eager.lens[steps % 2].tolist() == [budget, 12 + steps, budget]
