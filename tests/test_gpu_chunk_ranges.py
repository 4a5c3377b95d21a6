"""Chunk attention at the ends of binary32's range: values whose sums are just
finite.  Tolerances are test_gpu_chunk's."""
import numpy as np
import pytest

from test_gpu_chunk import BF16, Case, _f64

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
