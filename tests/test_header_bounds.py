"""What the headers promise about roundings, held against the roundings (no GPU):
a bound has to cover the worst case of a round to nearest, and be within a factor
of two of it (four for pairs: what the first rounding leaves is below its half
step, so that the second's half step is half the product of the two)."""
import os
import re

import pytest
import torch

from conftest import ROOT

F16, BF16 = torch.float16, torch.bfloat16


def _words(name, function):
    """The comment before a function's declaration, one space between words."""
    with open(os.path.join(ROOT, "include", name)) as f:
        text = f.read()
    text = text[:re.search(rf"QSA_API \w+ {function}\(", text).start()]
    return " ".join(text[text.rindex("/*"):].replace("\n *", " ").split())


def _powers(words, pattern):
    m = re.search(pattern, words)
    assert m, (pattern, words)
    return [2.0 ** -int(x) for x in m.groups()]


def _weights(top):
    """Weights from nothing up to `top`, ties and their neighbours among them."""
    g = torch.Generator().manual_seed(1)
    w = torch.exp2(-60 * torch.rand(400000, generator=g, dtype=torch.float64))
    ties = [(2 * i + 1) * 2.0 ** -12 + d for i in range(1025) for d in (-2.0 ** -23, 0.0, 2.0 ** -23)]
    ties += [1 + x + d for x in (2.0 ** -11, 2.0 ** -8, 3 * 2.0 ** -8) for d in (0.0, 2.0 ** -23)]
    ties = torch.tensor(ties, dtype=torch.float64)
    every = torch.cat([w] + [ties * 2.0 ** -k for k in range(0, 50)])
    return (every[every <= 1] * top).float()


def _off(w, dtype, pair):
    h = w.to(dtype)
    got = h.double()
    if pair:
        got = got + (w - h.float()).to(dtype).double()
    return (got - w.double()).abs()


def _hold(w, off, rel, least, total, within=2):
    """off <= max(rel * w, least * total), and not by far."""
    w = w.double()
    assert (off <= torch.maximum(rel * w, torch.full_like(w, least * total))).all()
    large = w * rel > least * total
    assert (off[large] / w[large]).max() > rel / within


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_chunk_attentions_weights(dtype):
    words = _words("qsa_chunk.h", "qsa_chunk_attention")
    a, b, c, d = _powers(
        words, r"off by at most 2\^-(\d+) of itself, or 2\^-(\d+) of its row's sum of weights where "
               r"that is more \(FP16, and any E4M3 cache\), 2\^-(\d+) or 2\^-(\d+) \(BF16\)")
    # the reference's own weight is in the sum: 2^8 of weights up to 2^15, 2^-8 of 1
    if dtype == F16:
        w = _weights(2.0 ** 15)
        _hold(w, _off(w, dtype, False), a, b, 2.0 ** 8)
    else:
        w = _weights(1.0)
        _hold(w, _off(w, dtype, False), c, d, 2.0 ** -8)
        assert d * 2.0 ** -8 >= 2.0 ** -126            # smaller weights are none


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_dense_attentions_weights(dtype):
    words = _words("qsa_cache.h", "qsa_paged_attention")
    pair = _powers(words, r"by 2\^-(\d+) \(FP16\) or 2\^-(\d+) \(BF16\) where")
    one = _powers(words, r"by 2\^-(\d+) \(FP16, and any E4M3 cache\) or 2\^-(\d+) \(BF16\) elsewhere")
    least, far, least_b = _powers(
        words, r"or by 2\^-(\d+) of the row's sum of weights \(FP16; logits past 2\^19: 2\^-(\d+)\), "
               r"2\^-(\d+) \(BF16\), where that is more")
    i = [F16, BF16].index(dtype)
    # the largest weight is 2^15 (FP16; less an eighth of a power where logits reach 2^19,
    # 1 at least wherever they are) or 1
    w = _weights(2.0 ** 15 if dtype == F16 else 1.0)
    for rel, two in ((pair[i], True), (one[i], False)):
        _hold(w, _off(w, dtype, two), rel, (least, least_b)[i], 2.0 ** 14.875 if dtype == F16 else 1.0,
              4 if two else 2)
    if dtype == F16:
        w = _weights(1.0)
        _hold(w, _off(w, dtype, False), one[i], far, 1.0)
    else:
        assert least_b >= 2.0 ** -126


def test_norms_sum_of_squares():
    # the least mean square that the header names, from squares that binary32 rounds to
    # multiples of 2^-149: off by less than its own rounding; and the elements that it says
    # are never too large
    words = _words("qsa_rope.h", "qsa_qk_norm_rope")
    assert "sum_j x_j^2 has to be finite there" in words
    least, = _powers(words, r"eps \+ \(sum_j x_j\^2\) / head_dim 2\^-(\d+) at least")
    large = float(2 ** int(re.search(r"elements up to 2\^(\d+)\)", words).group(1)))
    for dim in (8, 128, 256):
        for spread in (0.0, 8.0, 16.0):                      # elements of 2^-spread besides
            x = torch.full((dim,), 2.0 ** -spread, dtype=torch.float64)
            x[0] = 1.0
            x = (x * (least / (x * x).mean()).sqrt() * 1.01).to(BF16).float()
            exact = (x.double() ** 2).mean()
            got = (x * x).double().mean()
            assert exact >= least and (got / exact - 1).abs() <= 2.0 ** -24
        x = torch.full((dim,), large, dtype=torch.float32)
        assert (x * x).sum().isfinite()
    assert dim * (2.0 * large) ** 2 >= 2.0 ** 128            # twice as much would be
