"""Norms with rotation of rows whose sum of squares is at the ends of what
include/qsa_rope.h takes.  Tolerances are test_gpu_rope's."""
import pytest
import torch

import sparse_paged_attention_qsa_gb300 as qsa
from test_gpu_rope import BF16, DEV, _check, _freqs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [8, 64, 128, 256])
def test_rows_at_the_ends_of_the_sum(d, inter):
    g = torch.Generator(device=DEV).manual_seed(d)
    q = torch.empty((3, 40, d), device=DEV)
    big = torch.randint(0, 2, (3, 20, d), generator=g, device=DEV) * 2.0 - 1
    q[:, :10] = big[:, :10] * 2.0 ** 59                      # the largest elements of any row
    q[:, 10:20] = big[:, 10:] * 2.0 ** -60                   # a mean square of 2^-120
    q[:, 20:30] = torch.randn((3, 10, d), generator=g, device=DEV).clamp(-4, 4) * 2.0 ** 57
    # one element that is the mean square, the others' squares subnormal or gone
    q[:, 30:] = torch.randn((3, 10, d), generator=g, device=DEV) * 2.0 ** -70
    q[:, 30:, d // 2] = 2.0 ** -60 * d ** 0.5 * 1.01
    q = q.to(BF16)
    squares = q.double() ** 2
    assert squares.sum(-1).max() < 2.0 ** 128 and squares.mean(-1).min() >= 2.0 ** -120
    pos = torch.tensor([5, 4000, 77], device=DEV)
    f = _freqs(d // 16 * 16)
    for x in (q, q.sign() * 2.0 ** -133):                    # ... and any row where eps is as large
        eps = 0.0 if x is q else 2.0 ** -120
        z, _ = qsa.qsa_qk_norm_rope(x, None, pos, inv_freq=f if f.numel() else None, eps=eps,
                                    interleaved=inter)
        _check(z, x, None, pos, f, eps, inter)
