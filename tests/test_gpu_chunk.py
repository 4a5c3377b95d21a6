"""GPU parity of qsa_chunk_attention and qsa_prefix_attention
(include/qsa_chunk.h) against oracle/chunk.py, through the binding.

Tolerances (per element, from the arithmetic; S the entries a row sees):
  logit   |dz| <= D * 2^-23 * scale * sum |q k| (a binary32 dot of D exact
          products, each addition off by one unit of the running sum of
          magnitudes: the tensor core truncates; the scaling's two roundings are
          in it, D >= 64).  BF16 queries of an E4M3 cache enter as FP16 after a
          scaling of the row: elements below 2^-25 of its largest may be lost,
          D * 2^-24 * scale * max|q| max|k|;
  weight  relative 2|dz| (numerator and denominator) + 2^-20 (the exponential,
          the rescalings, the joins) + S * 2^-23, the additions of a sum;
  output  sum_e p_e |V_e| times (the weight's error + half a step of the type
          that the weights are rounded to, FP16 over an E4M3 cache, + S * 2^-23
          for the product's additions), + S * 2^-30 max|V| (FP16 weights below
          2^-14 of a sum's reference are subnormal), + half a step of the
          output's type times the value, + half its smallest subnormal;
  lse     |dz| + 2^-20 + S * 2^-23 + 2^-22 |lse|."""
import numpy as np
import pytest
import torch

import sparse_paged_attention_qsa_gb300 as qsa
from oracle import chunk as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134}


def _half(t):
    return torch.finfo(t).eps / 2


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
    """A batch over its own shuffled pages.  reqs: (new, cached before) of each."""

    def __init__(self, reqs, hq, hk, d, size, dtype=F16, cache=None, layout="split", window=0,
                 sink=0, prefix=None, seed=0, pad=(0, 0), scale=None):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        cpu = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        ctx = [n + old for n, old in reqs]
        cols = max(1, -(-max(ctx) // size))
        pcols = -(-(prefix or 0) // size)
        pages = len(reqs) * cols + pcols + 2
        self.k, self.v = make_cache(pages, size, hk, d, cache, layout, gen)
        ids = torch.randperm(pages, generator=cpu).to(torch.int32).to(DEV)
        self.tables = ids[:len(reqs) * cols].view(len(reqs), cols).clone()
        self.ptable = ids[len(reqs) * cols:len(reqs) * cols + pcols].clone()
        self.plen = torch.tensor([prefix or 0], dtype=torch.int32, device=DEV)
        self.prefix = prefix
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        starts = np.cumsum([0] + [n for n, _ in reqs]) + pad[0]
        self.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
        rows = int(starts[-1]) + pad[1]
        self.q = _values((rows, hq, d), dtype, gen)
        self.k_scale = self.v_scale = None
        if cache == E4M3:
            self.k_scale = 0.25 + torch.rand(hk, generator=gen, device=DEV)
            self.v_scale = 0.25 + torch.rand(hk, generator=gen, device=DEV)
        self.window, self.sink = window, sink
        self.scale = d ** -0.5 if scale is None else scale
        self.cache = cache

    def run(self, q=None, out=None, lse=True, **kw):
        q = self.q if q is None else q
        if out is None:
            out = torch.full(q.shape, 5.0, dtype=q.dtype, device=DEV)
        lse = torch.full(q.shape[:2], 6.0, device=DEV) if lse is True else lse
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        common = dict(scale=self.scale, k_scale=self.k_scale, v_scale=self.v_scale, out=out, lse=lse,
                      error_word=err, **kw)
        if self.prefix is None:
            qsa.qsa_chunk_attention(q, self.k, self.v, self.tables, self.starts, self.ctx,
                                    window=self.window, num_sink=self.sink, **common)
        else:
            qsa.qsa_prefix_attention(q, self.k, self.v, self.ptable, self.plen, self.tables,
                                     self.starts, self.ctx, **common)
        return out, lse, err

    def oracle(self):
        return K.attention(_f64(self.q), _f64(self.k), _f64(self.v), self.tables.cpu().numpy(),
                           self.starts.tolist(), self.ctx.tolist(), self.scale, self.window,
                           self.sink, self.ptable.tolist(), int(self.plen), _f64(self.k_scale),
                           _f64(self.v_scale))

    def check(self, out, lse, want=None):
        r = self.oracle() if want is None else want
        dt, d = out.dtype, self.q.shape[2]
        mine = r["mine"]
        got, vmax = _f64(out), np.nan_to_num(np.abs(_f64(self.v)), nan=0.0, posinf=0.0).max(initial=0)
        if self.v_scale is not None:
            vmax = vmax * float(self.v_scale.max())
        dz = d * 2.0 ** -23 * r["mag"]
        if self.cache == E4M3 and dt == BF16:
            dz = dz + d * 2.0 ** -24 * self.scale * np.abs(_f64(self.q)).max(initial=0) * \
                np.nan_to_num(np.abs(_f64(self.k))).max(initial=0) * float(self.k_scale.max())
        seen = r["seen"][:, None]
        rel = 2 * dz + 2.0 ** -20 + seen * 2.0 ** -23
        p_half = _half(F16 if self.cache == E4M3 else dt)
        tol = r["spread"] * (rel + p_half + seen * 2.0 ** -23)[..., None] + \
            (seen * 2.0 ** -30 * vmax)[..., None]
        tol = tol + _half(dt) * (np.abs(r["out"]) + tol) + TINY[dt]
        bad = np.abs(got - r["out"]) > tol
        bad |= ~np.isfinite(got)
        bad[~mine] = False
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - r["out"])[bad][:5], tol[bad][:5])
        assert (got[~mine] == 5.0).all()
        empty = mine & (r["seen"] == 0)
        assert (got[empty] == 0).all()
        if lse is not None:
            got = lse.double().cpu().numpy()
            assert (got[~mine] == 6.0).all() and (got[empty] == -np.inf).all()
            full = mine & (r["seen"] > 0)
            tol = (dz + 2.0 ** -20 + seen * 2.0 ** -23 + 2.0 ** -22 * np.abs(r["lse"]))[full]
            diff = np.abs(got[full] - r["lse"][full])
            assert (diff <= tol).all(), (diff - tol).max()
        return r


MIXED = [(1, 0), (1, 16), (3, 5), (0, 9), (40, 0), (129, 3), (1, 300), (8, 120), (0, 0), (70, 190)]


@pytest.mark.parametrize("prefix", [None, 0, 1, 150])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("hq,hk,d,size,layout", [
    (4, 2, 64, 16, "split"), (3, 1, 256, 512, "packed"), (8, 2, 128, 64, "heads"),
    (5, 1, 128, 8, "wide"), (6, 6, 64, 128, "packed"), (16, 1, 64, 32, "heads"), (2, 2, 256, 16, "wide")])
def test_mixed_batch(hq, hk, d, size, layout, dtype, cache, prefix):
    c = Case(MIXED, hq, hk, d, size, dtype, cache, layout, prefix=prefix, pad=(0, 3))
    out, lse, err = c.run()
    r = c.check(out, lse)
    assert int(err) == r["err"] == 0


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (BF16, E4M3)])
@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (5, 4), (64, 0), (100, 7), (128, 129),
                                         (3, 1000), (10 ** 12, 4), (0, 10 ** 12), (33, 200)])
def test_windows_and_sinks(window, sink, dtype, cache):
    reqs = [(1, 700), (1, 3), (200, 400), (9, 260), (300, 0), (130, 129), (2, 127)]
    c = Case(reqs, 6, 2, 64, 16, dtype, cache, window=window, sink=sink, seed=3, pad=(2, 2))
    out, lse, err = c.run()
    assert c.check(out, lse)["err"] == int(err) == 0


@pytest.mark.parametrize("d,size", [(64, 8), (128, 64), (256, 32)])
@pytest.mark.parametrize("window,sink", [(0, 0), (700, 3)])
def test_long_prompts_and_contexts(d, size, window, sink):
    # several row tiles, cut runs, and a single token at the end of a long context
    c = Case([(900, 1200), (1, 6000), (517, 0)], 4, 1, d, size, BF16, window=window, sink=sink, seed=4)
    out, lse, err = c.run()
    c.check(out, lse)
    c = Case([(1, 20000)], 4, 1, d, size, F16, window=window * 9, sink=sink, seed=5)
    out, lse, err = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("hq,hk,reqs,prefix", [
    (1, 1, [(1, 0)], 4000), (4, 1, [(1, 10)] * 40, 900), (20, 4, [(1, 3), (2, 0), (5, 77)], 2050),
    (3, 1, [(4, 100)] * 70, 1000), (8, 8, [(1, 0)] * 3, 5000), (4, 2, [(200, 0), (130, 0)], 640),
    (16, 1, [(0, 50), (1, 0), (0, 0)], 129)])
@pytest.mark.parametrize("d,dtype,cache", [(64, BF16, BF16), (128, F16, F16), (256, F16, F16),
                                           (128, BF16, E4M3)])
def test_prefix_batches(hq, hk, reqs, prefix, d, dtype, cache):
    c = Case(reqs, hq, hk, d, 16, dtype, cache, prefix=prefix, seed=6)
    out, lse, err = c.run()
    assert c.check(out, lse)["err"] == int(err) == 0


@pytest.mark.parametrize("prefix", [None, 37])
@pytest.mark.parametrize("d,dtype,cache", [(64, F16, F16), (128, BF16, BF16), (256, BF16, BF16),
                                           (128, F16, E4M3)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_hidden_entries_hold_does_not_matter(bad, d, dtype, cache, prefix):
    if cache == E4M3 and bad == bad:
        pytest.skip("E4M3 holds no infinities")
    reqs = [(40, 100), (1, 21), (150, 0), (6, 6)]
    window, sink = (0, 0) if prefix else (50, 3)
    c = Case(reqs, 4, 2, d, 32, dtype, cache, window=window, sink=sink, prefix=prefix, seed=7)
    clean, lse, _ = c.run()
    want = c.check(clean, lse)
    used = torch.zeros(c.k.shape[:2], dtype=torch.bool)      # entries that some row sees
    for b, (n, old) in enumerate(reqs):
        for e in range(n + old):
            if not window or e >= old + 1 - window or e < sink:
                used[int(c.tables[b, e // 32]), e % 32] = True
    for e in range(prefix or 0):
        used[int(c.ptable[e // 32]), e % 32] = True
    used = used.to(DEV)
    for x in (c.k, c.v):
        y = x.float()
        y[~used] = bad
        x.copy_(y.to(x.dtype)) if cache == E4M3 else x.copy_(y)
    out, lse2, _ = c.run()
    assert torch.equal(out, clean) and torch.equal(lse2, lse)
    # an entry of a later token: the rows before it do not see it
    last = reqs[2][0] - 1
    page, slot = int(c.tables[2, last // 32]), last % 32
    c.k[page, slot] = torch.full((2, d), bad, device=DEV).to(c.k.dtype)
    c.v[page, slot] = torch.full((2, d), bad, device=DEV).to(c.v.dtype)
    out, lse3, _ = c.run()
    row = int(c.starts[3]) - 1
    keep = [i for i in range(len(want["mine"])) if i != row]
    assert out[keep].isfinite().all()
    got = out.clone()
    got[row], lse3[row] = clean[row], lse[row]
    c.check(got, lse3, want)
    assert not out[row].isfinite().any()


def test_bad_pages_long_contexts_and_empty_rows():
    for prefix in (None, 100):
        c = Case([(5, 60), (1, 40), (3, 0), (2, 10), (1, 0)], 4, 2, 64, 16, prefix=prefix, seed=8)
        c.tables[0, 1] = -1
        c.tables[1, 2] = 10 ** 9
        c.ctx[2] = 1                                         # two of three rows see nothing
        c.ctx[3] = 500                                       # past the table
        c.ctx[4] = -7
        if prefix:
            c.ptable[3] = -5
        out, lse, err = c.run()
        r = c.check(out, lse)
        assert int(err) == r["err"] == K.DERR_KV_PAGE | K.DERR_CONTEXT
    c = Case([(3, 4)], 2, 1, 128, 16, prefix=20, seed=9)
    c.plen.fill_(1000)
    out, lse, err = c.run()
    r = c.check(out, lse)
    assert int(err) == r["err"] == K.DERR_CONTEXT
    c.plen.fill_(-3)
    out, lse, err = c.run()
    assert c.check(out, lse)["err"] == int(err) == 0
    c.plen.fill_(9)                                          # and none to look up
    c.ptable = c.ptable[:0]
    out, lse, err = c.run()
    assert c.check(out, lse)["err"] == int(err) == K.DERR_CONTEXT
    # fewer entries than new tokens, a window wider than any context
    for window in (2 ** 31 - 1, 2 ** 40):
        c = Case([(300, 0), (1, 50)], 4, 2, 64, 16, window=window, sink=2, seed=9)
        c.ctx[0] = 40
        out, lse, err = c.run()
        assert c.check(out, lse)["err"] == int(err) == 0
    # no pages at all
    c = Case([(2, 3)], 2, 1, 64, 16, seed=9)
    c.k, c.v = c.k[:0], c.v[:0]
    out, lse, err = c.run()
    assert (out == 0).all() and (lse == -float("inf")).all() and int(err) == K.DERR_KV_PAGE


@pytest.mark.parametrize("starts", [[0, 5, 3, 20], [-4, 2, 9, 9], [9, 9, 9, 9], [0, 0, 50, 60], [7, 3, 1, 0],
                                    [-2 ** 31, 0, 4, 2 ** 31 - 1], [2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31, 5]])
def test_malformed_starts_stay_inside(starts):
    # what such rows hold is undefined; nothing outside the arrays is touched
    for prefix in (None, 40):
        c = Case([(4, 30), (4, 60), (4, 0)], 4, 2, 64, 16, prefix=prefix, seed=10)
        c.starts = torch.tensor(starts, dtype=torch.int64).to(torch.int32).to(DEV)
        big = torch.full((c.q.shape[0] + 2, 4, 64), 5.0, dtype=F16, device=DEV)
        out, lse, _ = c.run(out=big[1:-1])
        torch.cuda.synchronize()
        assert (big[0] == 5).all() and (big[-1] == 5).all()
        c = Case([(4, 30), (4, 60), (4, 0)], 4, 2, 64, 16, prefix=prefix, seed=10)
        c.check(*c.run()[:2])                                # and the next call is right


@pytest.mark.parametrize("mul", [1e-6, 30.0, 3e4, 1e12])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scales_of_any_size(mul, dtype):
    c = Case([(40, 200), (1, 500)], 4, 2, 64, 16, dtype, scale=mul, seed=11)
    # small whole numbers: every logit is exact before the scale, so that large
    # scales keep the softmax's winners
    c.q.copy_(c.q.float().round().clamp(-3, 3)), c.k.copy_(c.k.float().round().clamp(-3, 3))
    out, lse, _ = c.run()
    assert out.isfinite().all()
    z = np.float64(np.float32(np.float64(np.float32(mul)) * 1.4426950408889634)) * np.log(2.0)
    c.scale = float(z)
    c2 = c.oracle()
    c2["mag"] = c2["mag"] * 2.0 ** -6                        # one rounding of the scaled value at most
    big = c2["mag"].max() * 64 * 2.0 ** -23
    if big < 0.5:
        c.check(out, lse, c2)
    else:                                                    # one-hot rows: equal maxima share
        c2["mag"][:] = 0
        c.check(out, None, c2)


@pytest.mark.parametrize("hq,hk,reqs", [
    (4, 2, [(200, 1300)]), (4, 2, [(1, 1500)]), (4, 2, [(20, 700), (3, 1200), (1, 250)]),
    (16, 8, [(128, 1400)] * 4), (8, 8, [(1, 1700)] * 64)])     # long runs of each mode
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, E4M3)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_maxima_that_move_at_every_tile(d, dtype, cache, hq, hk, reqs):
    # logits that rise by 12 every 128 entries: the sums so far are rescaled each time
    c = Case(reqs, hq, hk, d, 64, dtype, cache, scale=12.0, seed=19)
    c.q.mul_(2.0 ** -6)
    c.q[..., 0] = 1
    k = c.k.float()
    for b, (n, old) in enumerate(reqs):
        e = torch.arange(n + old, device=DEV)
        k[c.tables[b].long()[e // 64], e % 64, :, 0] = (e // 128).float()[:, None]
    c.k.copy_(k.to(cache))
    if cache == E4M3:
        c.k_scale.fill_(1.0)
    out, lse, err = c.run()
    c.check(out, lse)
    assert int(err) == 0


def test_equal_logits_far_up_share_evenly():
    # logits of 2^30 and more: their reference is a binary32 value of its own
    c = Case([(1, 99)], 1, 1, 64, 16, F16, scale=1e9, seed=12)
    c.q.fill_(1.0), c.k.fill_(1.0)
    out, _, _ = c.run()
    pages = c.tables[0].long()
    mean = c.v[pages].flatten(0, 1)[:100, 0].double().mean(0)
    assert (out[0, 0].double() - mean).abs().max() < 2e-3


def test_strides_streams_repeats_and_optional_lse():
    c = Case([(33, 50), (1, 200), (90, 0)], 8, 2, 128, 32, BF16, seed=13)
    out, lse, _ = c.run()
    want = c.check(out, lse)
    rows = c.q.shape[0]
    wide = torch.full((rows, 12, 144), 5.0, dtype=BF16, device=DEV)
    q = torch.zeros((8, rows + 2, 136), dtype=BF16, device=DEV)[:, 1:-1, :128].transpose(0, 1)
    q.copy_(c.q)
    o2, l2, _ = c.run(q=q, out=wide[:, 2:10, :128])
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert (wide[:, :2] == 5).all() and (wide[:, 10:] == 5).all() and (wide[..., 128:] == 5).all()
    o3, _, _ = c.run(lse=None)
    assert torch.equal(o3, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o4, l4, _ = c.run(stream=side)
    side.synchronize()
    assert torch.equal(o4, out) and torch.equal(l4, lse)
    ws = torch.empty(max(256, qsa.qsa_chunk_attention_workspace_bytes(
        c.k, c.v, c.tables, num_tokens=rows, num_heads=8)), dtype=torch.uint8, device=DEV)
    for fill in (0, 255):
        ws.fill_(fill)
        o5, l5, _ = c.run(workspace=ws)
        assert torch.equal(o5, out) and torch.equal(l5, lse)
    c.check(o5, l5, want)


@pytest.mark.parametrize("prefix", [None, 500])
def test_graphs_that_share_a_workspace_and_change_lengths(prefix):
    cases = [Case([(20, 100), (1, 300), (3, 40)], 4, 1, 128, 16, F16, prefix=prefix, seed=s)
             for s in (14, 15)]
    eager = [c.run()[:2] for c in cases]
    need = qsa.qsa_chunk_attention_workspace_bytes(
        cases[0].k, cases[0].v, cases[0].tables, num_tokens=24, num_heads=4,
        prefix_cols=-1 if prefix is None else cases[0].ptable.shape[0])
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for c in cases:
        out, lse = torch.zeros_like(eager[0][0]), torch.zeros_like(eager[0][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=out, lse=lse, workspace=ws)
        graphs.append(g), outs.append((out, lse))
    for _ in range(3):
        for g, o, e in zip(graphs, outs, eager):
            o[0].zero_()
            g.replay()
            assert torch.equal(o[0], e[0]) and torch.equal(o[1], e[1])
    # other lengths in the same buffers
    c = cases[0]
    c.ctx.copy_(torch.tensor([20, 250, 3], device=DEV, dtype=torch.int32))
    c.starts.copy_(torch.tensor([0, 2, 20, 24], device=DEV, dtype=torch.int32))
    graphs[0].replay()
    c.check(*outs[0])


def test_offsets_past_32_bits():
    # a pool of more than 2^32 bytes and elements, its last pages in use
    d, size, pages = 128, 64, 300000
    k = torch.empty((pages, size, 1, d), dtype=F16, device=DEV)
    v = torch.empty((pages, size, 1, d), dtype=F16, device=DEV)
    assert k.numel() > 2 ** 31 and k.numel() * 2 > 2 ** 32
    c = Case([(70, 200), (1, 300)], 4, 1, d, size, F16, seed=16)
    ids = torch.tensor([pages - 1 - 7 * i for i in range(c.k.shape[0])], device=DEV)
    k[ids], v[ids] = c.k, c.v
    want, lse, _ = c.run()
    c.check(want, lse)
    c.k, c.v, c.tables = k, v, ids[c.tables.long()].to(torch.int32)
    out, lse2, err = c.run()
    assert torch.equal(out, want) and torch.equal(lse2, lse) and int(err) == 0


@pytest.mark.parametrize("hq,hk", [(130, 1), (131, 1), (256, 2), (300, 1), (96, 1), (40, 8)])
def test_groups_of_any_width(hq, hk):
    for prefix, reqs in ((None, [(3, 40), (1, 200), (5, 0)]), (70, [(2, 9), (1, 0)])):
        c = Case(reqs, hq, hk, 64, 16, BF16, prefix=prefix, seed=20)
        out, lse, err = c.run()
        assert c.check(out, lse)["err"] == int(err) == 0


@pytest.mark.parametrize("cache", [F16, E4M3])
def test_pages_that_no_row_sees_may_be_gone(cache):
    reqs = [(1, 900), (40, 600), (1, 33)]
    c = Case(reqs, 4, 2, 64, 16, F16, cache, window=100, sink=20, seed=21)
    out, lse, err = c.run()
    want = c.check(out, lse)
    for b, (n, old) in enumerate(reqs):
        for col in range(c.tables.shape[1]):
            seen = any(e < old + n and (e >= old + 1 - 100 or e < 20) for e in range(col * 16, col * 16 + 16))
            if not seen:
                c.tables[b, col] = -1
    out2, lse2, err = c.run()
    assert torch.equal(out2, out) and torch.equal(lse2, lse) and int(err) == 0
    c.check(out2, lse2, want)


def test_two_streams_at_once():
    cases = [Case([(300, 200), (1, 900), (2, 7)], 4, 1, 128, 16, F16, seed=22),
             Case([(1, 3000)] * 20, 8, 2, 64, 32, BF16, prefix=400, seed=23)]
    want = [c.run()[:2] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(c.run()[:2])
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


def test_many_requests():
    g = torch.Generator().manual_seed(17)
    reqs = [(int(a), int(b)) for a, b in zip(torch.randint(0, 3, (3000,), generator=g),
                                             torch.randint(0, 40, (3000,), generator=g))]
    for prefix in (None, 70):
        c = Case(reqs, 2, 1, 64, 16, F16, prefix=prefix, seed=18)
        out, lse, err = c.run()
        c.check(out, lse)


def test_a_layers_operators_together():
    """A prompt in two parts, then single tokens: rotation, append, attention with a window and
    sinks; every token's row as the dense definition over the whole sequence has it."""
    hq, hk, d, size, total = 6, 2, 128, 16, 150
    gen = torch.Generator(device=DEV).manual_seed(19)
    x = _values((total, hq + 2 * hk, d), BF16, gen)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).to(BF16), None
    freq = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).to(DEV, torch.float32)
    k_cache, v_cache = make_cache(12, size, hk, d, BF16, "packed", gen)
    k_cache.fill_(float("nan")), v_cache.fill_(float("nan"))
    tables = torch.randperm(12, generator=gen, device=DEV)[:10].view(1, 10).to(torch.int32)
    out = torch.zeros((total, hq, d), dtype=BF16, device=DEV)
    at = 0
    for n in [90, 50] + [1] * 10:
        part = x[at:at + n]
        pos = torch.arange(at, at + n, device=DEV)
        q, k = qsa.qsa_qk_norm_rope(part[:, :hq], part[:, hq:hq + hk], pos, wq, wk, inv_freq=freq)
        qsa.qsa_paged_append(k, part[:, hq + hk:], k_cache, v_cache, tables,
                             torch.zeros(n, dtype=torch.int32, device=DEV), pos)
        at += n
        qsa.qsa_chunk_attention(q, k_cache, v_cache, tables,
                                torch.tensor([0, n], dtype=torch.int32, device=DEV),
                                torch.tensor([at], dtype=torch.int32, device=DEV), window=40,
                                num_sink=4, out=out[at - n:at])
    z = K.norm_rope(_f64(x[:, :hq + hk]), None, range(total), _f64(freq), 1e-6, False)
    q = K.norm_rope(_f64(x[:, :hq]), _f64(wq), range(total), _f64(freq), 1e-6, False)
    k, v = z[:, hq:], _f64(x[:, hq + hk:])
    for t in (0, 3, 39, 40, 44, 89, 90, 139, 140, 149):
        e = np.array([i for i in range(t + 1) if t - i < 40 or i < 4])
        for h in range(hq):
            s = d ** -0.5 * (k[e, h // 3] @ q[t, h])
            p = np.exp(s - s.max())
            want = (p / p.sum()) @ v[e, h // 3]
            # q and k are rounded to BF16 on the way: logits off by their rounding
            dz = 2 * 2.0 ** -9 * d ** -0.5 * (np.abs(k[e, h // 3]) @ np.abs(q[t, h])).max()
            bound = (p / p.sum()) @ np.abs(v[e, h // 3]) * (2 * dz + 2 * 2.0 ** -9 + 2.0 ** -12)
            assert (np.abs(_f64(out[t, h]) - want) <= bound + 2.0 ** -9 * np.abs(want)).all()
