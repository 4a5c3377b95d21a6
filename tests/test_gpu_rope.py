"""GPU parity of qsa_qk_norm_rope (include/qsa_rope.h) against oracle/chunk.py.

Tolerance of an element z of a pair (y_a, y_b), u = 2^-24: the norm's factor is
off by 13 additions, a square root, a division and three products (relative
2^-19 covers 20 u twice over), the angle by 2^-24 of a half turn, sine and
cosine by two units (2^-22), the turn by three roundings, all of at most |y_a| +
|y_b|: 2^-18 of that together, + half a step of the type, relative to z, + half
its smallest subnormal."""
import numpy as np
import pytest
import torch

import sparse_paged_attention_qsa_gb300 as qsa
from oracle import chunk as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16
HALF_STEP = {F16: torch.finfo(F16).eps / 2, BF16: torch.finfo(BF16).eps / 2}
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134}


def _f64(t):
    return t.float().double().cpu().numpy()


def _freqs(rot, base=1e4):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).to(DEV, torch.float32)


def _check(got, x, w, pos, f, eps, inter, before=None):
    want = K.norm_rope(_f64(x), None if w is None else _f64(w), pos.tolist(), _f64(f), eps, inter)
    flat = K.norm_rope(_f64(x), None if w is None else _f64(w), pos.tolist(), _f64(f)[:0], eps, inter)
    mag = np.abs(flat)
    half = f.numel()
    a = 2 * np.arange(half) if inter else np.arange(half)
    b = a + 1 if inter else a + half
    both = mag[..., a] + mag[..., b]
    mag[..., a] = mag[..., b] = both
    live = pos.cpu().numpy() >= 0
    err = np.abs(_f64(got) - want)[live]
    tol = (2.0 ** -18 * mag + HALF_STEP[got.dtype] * (np.abs(want) + 2.0 ** -18 * mag) +
           TINY[got.dtype])[live]
    assert (err <= tol).all(), (err - tol).max()
    if before is not None:
        assert torch.equal(got[~torch.from_numpy(live).to(DEV)], before[~torch.from_numpy(live).to(DEV)])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,hq,hk,d,rot", [
    (1, 3, 1, 256, 64), (1, 1, 1, 8, 0), (2, 5, 3, 16, 16), (7, 4, 2, 64, 64), (33, 32, 8, 128, 128),
    (5, 9, 1, 80, 32), (3, 2, 2, 96, 96), (19, 6, 6, 192, 96), (300, 3, 1, 256, 256), (4, 70, 7, 24, 16),
    (6, 2, 1, 248, 240), (1000, 1, 1, 64, 32), (2, 300, 40, 32, 32)])
def test_against_the_oracle(tokens, hq, hk, d, rot, dtype, inter):
    g = torch.Generator(device=DEV).manual_seed(tokens * 31 + d)
    q = torch.randn((tokens, hq, d), generator=g, device=DEV).to(dtype)
    k = (torch.randn((tokens, hk, d), generator=g, device=DEV) * 5).to(dtype)
    w = [(1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(dtype) for _ in range(2)]
    pos = torch.randint(-1, 200000, (tokens,), generator=g, device=DEV)
    if tokens == 1:
        pos[0] = 77777
    f = _freqs(rot)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 8.0)
    r = qsa.qsa_qk_norm_rope(q, k, pos, *w, inv_freq=f if rot else None, interleaved=inter, eps=1e-5,
                             q_out=qo, k_out=ko)
    assert r[0] is qo and r[1] is ko
    _check(qo, q, w[0], pos, f, 1e-5, inter, torch.full_like(q, 7.0))
    _check(ko, k, w[1], pos, f, 1e-5, inter, torch.full_like(k, 8.0))
    # results of its own, binary32 weights, one of them absent
    q2, k2 = qsa.qsa_qk_norm_rope(q, k, pos.abs(), w[0].float(), None, inv_freq=f if rot else None,
                                  interleaved=inter, eps=0.0)
    _check(q2, q, w[0], pos.abs(), f, 0.0, inter)
    _check(k2, k, None, pos.abs(), f, 0.0, inter)


def test_far_positions_and_any_frequency():
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 31 - 1, 2 ** 31 + 5, 2 ** 36 - 7], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn((len(pos), 2, 64), generator=g, device=DEV).to(F16)
    f = torch.tensor([1.0, 0.999999, 3.1415927, 6.2831855, 100.25, 1e-4, 1e-7, 1e-12, 1e-30, 0.0,
                      -0.5, -1e-3, 2.0 ** -40, 0.1, 1e-38, 7.0], device=DEV)
    for inter in (False, True):
        z, _ = qsa.qsa_qk_norm_rope(q, None, pos, inv_freq=f, interleaved=inter)
        _check(z, q, None, pos, f, 1e-6, inter)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_in_place_on_a_projections_rows(dtype):
    t, hq, hk, d = 37, 5, 2, 128
    x = torch.randn((t, hq + 2 * hk, d), device=DEV).to(dtype)
    before = x.clone()
    pos = torch.arange(t, device=DEV) * 100
    f = _freqs(d)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    qsa.qsa_qk_norm_rope(q, k, pos, inv_freq=f, q_out=q, k_out=k)
    _check(q, before[:, :hq], None, pos, f, 1e-6, False)
    _check(k, before[:, hq:hq + hk], None, pos, f, 1e-6, False)
    assert torch.equal(x[:, hq + hk:], before[:, hq + hk:])       # the values beside them
    # strides of every kind: heads outermost, gaps
    y = torch.randn((hq, t + 3, d + 8), device=DEV).to(dtype)[:, 1:t + 1, :d].transpose(0, 1)
    o = torch.zeros((t, 2 * hq, d), device=DEV, dtype=dtype)
    qsa.qsa_qk_norm_rope(y, None, pos, inv_freq=f, q_out=o[:, ::2])
    _check(o[:, ::2], y, None, pos, f, 1e-6, False)
    assert (o[:, 1::2] == 0).all()


def test_large_small_zero_and_not_finite_rows():
    d = 64
    q = torch.ones((1, 8, d), device=DEV, dtype=BF16)
    q[0, 0] = 0
    q[0, 1] = 2.0 ** -60
    q[0, 2] = 2.0 ** 60
    q[0, 3, 5] = float("inf")
    q[0, 4, 5] = float("nan")
    q[0, 5, 1:] = 0
    pos = torch.tensor([3], device=DEV)
    f = _freqs(d)
    z, _ = qsa.qsa_qk_norm_rope(q, None, pos, inv_freq=f, eps=1e-6)
    keep = [0, 1, 2, 5, 6, 7]
    _check(z[:, keep], q[:, keep], None, pos, f, 1e-6, False)
    assert z[0, 4].isnan().all() and z[0, 3, 5].isnan()
    assert (z[0, 3, [0, 1, 63]] == 0).all()             # elsewhere divided by an infinite norm


def test_streams_graphs_and_no_tokens():
    t, d = 64, 128
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn((t, 8, d), generator=g, device=DEV).to(BF16)
    k = torch.randn((t, 2, d), generator=g, device=DEV).to(BF16)
    pos, f = torch.arange(t, device=DEV), _freqs(d)
    want = qsa.qsa_qk_norm_rope(q, k, pos, inv_freq=f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qsa.qsa_qk_norm_rope(q, k, pos, inv_freq=f, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    x, y, p = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(pos)
    with torch.cuda.graph(graph):
        got = qsa.qsa_qk_norm_rope(x, y, p, inv_freq=f)
    for _ in range(2):
        x.copy_(q), y.copy_(k), p.copy_(pos)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        x.zero_(), y.zero_()
    a, b = qsa.qsa_qk_norm_rope(q[:0], k[:0], pos[:0], inv_freq=f)
    assert a.shape == (0, 8, d) and b.shape == (0, 2, d)
