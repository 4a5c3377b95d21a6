"""Chunk attention at the ends of binary32's range: values whose sums are just
finite, and queries whose logits' factor (over E4M3 caches a power of two for
each row is part of it) is not.  Tolerances are test_gpu_chunk's."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import BF16, E4M3, Case, _f64

pytestmark = pytest.mark.gpu

# row tiles of two halves, single tokens (split for heads of 64), runs that are cut, a
# prefix; enough of the first two that runs hold whole row tiles
BATCHES = [([(200, 500)] * 24, None), ([(1, 1700), (20, 300)] * 60, None), ([(1, 20000)], None),
           ([(1, 40), (3, 0), (70, 90)], 900)]


@pytest.mark.parametrize("reqs,prefix", BATCHES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_whose_sum_is_just_finite(d, reqs, prefix):
    # first entries of logit 0, one whose value is 2^126 with a logit of 5.5 (weights
    # 2^7.9 of the first ones', so that a reference need not move), three that fill the sum
    c = Case(reqs, 8, 4, d, 16, BF16, prefix=prefix, scale=1.0, seed=40)
    c.q.mul_(2.0 ** -6)
    c.q[..., 0] = 1
    c.k[..., 0] = 0
    last = [(c.tables[b], n + old) for b, (n, old) in enumerate(reqs) if old]
    if prefix:
        last = [(c.ptable, prefix)]
    for table, count in last:
        for e, z, v in ((count // 2, 5.5, 2.0 ** 126), (count // 3, 5.5, -2.0 ** 125),
                        (count // 4, 0.0, 2.0 ** 126), (3, 0.0, 2.0 ** 124)):
            page, slot = int(table[e // 16]), e % 16
            c.k[page, slot, :, 0], c.v[page, slot] = z, v
    out, lse, err = c.run()
    assert int(err) == 0
    c.check(out, lse)
    assert np.abs(_f64(out)).max() > 2.0 ** 110


FEW = [([(200, 500)], None), ([(1, 1700), (20, 300)] * 20, None)] + BATCHES[2:]


def _e4m3(reqs, prefix, d, scale=None):
    return Case(reqs, 4, 2, d, 16, BF16, E4M3, prefix=prefix, scale=scale, seed=41)


@pytest.mark.parametrize("reqs,prefix", FEW)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_tiny_queries_and_scales_of_an_e4m3_cache(d, reqs, prefix):
    # logits of 2^-170 and less: every entry weighs the same
    c = _e4m3(reqs, prefix, d)
    c.q.mul_(2.0 ** -110)
    c.k_scale.fill_(2.0 ** -64)
    out, lse, err = c.run()
    c.check(out, lse)
    assert int(err) == 0
    # ... beside rows of zeros, and rows of ordinary size
    c = _e4m3(reqs, prefix, d)
    c.q[::2] = 0
    c.q[1::4].mul_(2.0 ** -120)
    out, lse, err = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("reqs,prefix", FEW)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_huge_queries_of_an_e4m3_cache(d, reqs, prefix):
    # the row's largest element meets zeros alone
    c = _e4m3(reqs, prefix, d, scale=4.0)
    k = c.k.float()
    k[:] = 0
    c.k.copy_(k.to(E4M3))
    c.q.mul_(2.0 ** 118)
    c.k_scale.fill_(2.0 ** 40)
    out, lse, err = c.run()
    c.check(out, lse)
    assert int(err) == 0
    # equal logits of 2^109: lse is theirs
    k[..., 1] = 2.0 ** -9
    c.k.copy_(k.to(E4M3))
    c.k_scale.fill_(2.0 ** 20)
    c.q.zero_()
    c.q[..., 0], c.q[..., 1] = 2.0 ** 120, 2.0 ** 96
    out2, lse2, _ = c.run()
    assert torch.equal(out2, out)
    assert (lse2.double() - 2.0 ** 109).abs().max() <= 2.0 ** (109 - 22)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_subnormal_queries_of_an_e4m3_cache(d):
    # elements below 2^-126, a scale that makes their logits ordinary ones
    c = _e4m3([(20, 300), (1, 1700)], None, d, scale=2.0 ** 126)
    c.q.copy_((c.q.float().clamp(-3, 3) * 16).round() * 2.0 ** -133)
    assert float(c.q.float().abs().max()) < 2.0 ** -126
    out, lse, err = c.run()
    c.check(out, lse)
    assert np.abs(_f64(lse) - np.log(300)).max() > 0.02
