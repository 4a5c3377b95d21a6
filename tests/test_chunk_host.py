"""Host-side checks of qsa_qk_norm_rope, qsa_chunk_attention and
qsa_prefix_attention (no GPU): every bad argument is refused before any CUDA
call, so fake, never dereferenced device addresses are enough."""
import ctypes

import pytest
import torch

import sparse_paged_attention_qsa_gb300 as qsa
from sparse_paged_attention_qsa_gb300 import binding
from sparse_paged_attention_qsa_gb300 import build as qbuild

NULL, DTYPE, SHAPE, STRIDE, ALIGN, CONTRACT, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 6, 7, 8
CACHE = "k v pages size heads dim ks0 ks1 ks2 ks3 vs0 vs1 vs2 vs3 kscale vscale bt reqs cols bts0 dtype"


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load_library()


def _addr(k):
    return (1 << 36) * (k + 1)


def _arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _rope(lib, **over):
    a = dict(q=_addr(1), k=_addr(2), dt=2, tokens=10, hq=4, hk=2, dim=64, qs=(256, 64, 1),
             ks=(128, 64, 1), qw=_addr(3), kw=_addr(4), wdt=2, eps=1e-6, pos=_addr(5),
             freq=_addr(6), rot=64, inter=0, qo=_addr(7), ko=_addr(8), qos=(256, 64, 1),
             kos=(128, 64, 1))
    a.update(over)
    return lib.qsa_qk_norm_rope(
        a["q"], a["k"], a["dt"], a["tokens"], a["hq"], a["hk"], a["dim"], _arr(*a["qs"]),
        _arr(*a["ks"]), a["qw"], a["kw"], a["wdt"], a["eps"], a["pos"], a["freq"], a["rot"],
        a["inter"], a["qo"], a["ko"], _arr(*a["qos"]), _arr(*a["kos"]), None)


@pytest.mark.parametrize("over,want", [
    (dict(dt=3), DTYPE), (dict(dt=6), DTYPE), (dict(wdt=1), DTYPE), (dict(wdt=0), DTYPE),
    (dict(dim=60), SHAPE), (dict(dim=0), SHAPE), (dict(dim=264), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(tokens=1 << 31), SHAPE), (dict(hq=-1), SHAPE), (dict(hk=65537), SHAPE),
    (dict(rot=80), SHAPE), (dict(rot=8), SHAPE), (dict(rot=-16), SHAPE),
    (dict(eps=-1.0), CONTRACT), (dict(eps=float("nan")), CONTRACT), (dict(eps=float("inf")), CONTRACT),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(qo=0), NULL), (dict(ko=0), NULL), (dict(pos=0), NULL),
    (dict(freq=0), NULL),
    (dict(qs=(256, 64, 2)), STRIDE), (dict(qs=(260, 64, 1)), STRIDE), (dict(qs=(256, 0, 1)), STRIDE),
    (dict(ks=(128, 60, 1)), STRIDE), (dict(qos=(192, 64, 1)), STRIDE), (dict(kos=(64, 64, 1)), STRIDE),
    (dict(qos=(-256, 64, 1)), STRIDE), (dict(qs=(1 << 39, 64, 1)), STRIDE),
    (dict(q=_addr(1) + 8), ALIGN), (dict(ko=_addr(8) + 2), ALIGN), (dict(pos=_addr(5) + 4), ALIGN),
    (dict(freq=_addr(6) + 2), ALIGN), (dict(qw=_addr(3) + 1), ALIGN),
    (dict(kw=_addr(4) + 2, qw=_addr(3), wdt=3), ALIGN),
    (dict(qo=_addr(1) + 512), ALIAS),                   # q, a row further
    (dict(qo=_addr(1), qos=(512, 64, 1)), ALIAS),       # q, other strides
    (dict(qo=_addr(2)), ALIAS), (dict(ko=_addr(1)), ALIAS), (dict(ko=_addr(7)), ALIAS),
    (dict(qo=_addr(5) - 64), ALIAS), (dict(ko=_addr(6)), ALIAS), (dict(qo=_addr(3)), ALIAS),
    # a projection's rows [q | k] in place: k's heads inside q's
    (dict(qs=(512, 64, 1), qos=(512, 64, 1), qo=_addr(1), k=_addr(1) + 256, ks=(512, 64, 1)), ALIAS),
    # rows side by side, the last head of k over the next token's q
    (dict(qs=(384, 64, 1), qos=(384, 64, 1), qo=_addr(1), k=_addr(1) + 640, ks=(384, 64, 1)), ALIAS),
])
def test_rope_refuses(lib, over, want):
    assert _rope(lib, **over) == want


def test_rope_no_ops(lib):
    assert _rope(lib, tokens=0, q=0, k=0, qo=0, ko=0, pos=0) == 0
    assert _rope(lib, hq=0, hk=0) == 0


def _cache(a):
    return binding._CACHE.pack(*[a[f] for f in CACHE.split()])


def _attend(lib, prefix=False, query=False, **over):
    a = dict(k=_addr(1), v=_addr(2), pages=64, size=16, heads=2, dim=64, ks0=2048, ks1=128, ks2=64,
             ks3=1, vs0=2048, vs1=128, vs2=64, vs3=1, kscale=0, vscale=0, bt=_addr(3), reqs=4,
             cols=8, bts0=8, dtype=1,
             pt=_addr(4), pcols=5, plen=_addr(5), q=_addr(6), dt=1, tokens=12, hq=4, qs=(256, 64, 1),
             starts=_addr(7), ctx=_addr(8), scale=0.125, window=0, sink=0, out=_addr(9),
             os=(256, 64, 1), lse=_addr(10), ws=_addr(11), wsb=1 << 40, err=0)
    a.update(over)
    c = _cache(a)
    if query:
        return lib.qsa_chunk_attention_workspace_bytes(c, a["tokens"], a["hq"],
                                                       a["pcols"] if prefix else -1)
    tail = (a["out"], _arr(*a["os"]), a["lse"], a["ws"], a["wsb"], a["err"], None)
    head = (a["q"], a["dt"], a["tokens"], a["hq"], _arr(*a["qs"]), a["starts"], a["ctx"], a["scale"])
    if prefix:
        return lib.qsa_prefix_attention(c, a["pt"], a["pcols"], a["plen"], *head, *tail)
    return lib.qsa_chunk_attention(c, *head, a["window"], a["sink"], *tail)


BAD = [
    (dict(dim=96), SHAPE), (dict(size=12), SHAPE), (dict(heads=0), SHAPE), (dict(dtype=3), DTYPE),
    (dict(kscale=_addr(20)), CONTRACT), (dict(ks1=64), STRIDE), (dict(k=_addr(1) + 8), ALIGN),
    (dict(dt=2), DTYPE), (dict(dt=6), DTYPE), (dict(scale=0.0), CONTRACT),
    (dict(scale=float("inf")), CONTRACT), (dict(scale=-1.0), CONTRACT),
    (dict(scale=float("nan")), CONTRACT), (dict(tokens=-1), SHAPE), (dict(tokens=16777217), SHAPE),
    (dict(tokens=16777216, hq=128), SHAPE), (dict(hq=3), SHAPE), (dict(hq=0), SHAPE),
    (dict(hq=65536), SHAPE), (dict(qs=(256, 64, 2)), STRIDE), (dict(qs=(258, 64, 1)), STRIDE),
    (dict(os=(128, 64, 1)), STRIDE), (dict(os=(0, 64, 1)), STRIDE), (dict(q=0), NULL),
    (dict(out=0), NULL), (dict(starts=0), NULL), (dict(ctx=0), NULL), (dict(q=_addr(6) + 8), ALIGN),
    (dict(out=_addr(9) + 4), ALIGN), (dict(starts=_addr(7) + 2), ALIGN), (dict(lse=_addr(10) + 1), ALIGN),
    (dict(err=_addr(12) + 1), ALIGN), (dict(out=_addr(6)), ALIAS), (dict(out=_addr(1)), ALIAS),
    (dict(lse=_addr(8)), ALIAS), (dict(lse=_addr(9)), ALIAS), (dict(err=_addr(7) + 16), ALIAS),
    (dict(out=_addr(3) - 64), ALIAS), (dict(ws=0), WORKSPACE), (dict(wsb=1000), WORKSPACE),
    (dict(ws=_addr(11) + 128), ALIGN), (dict(ws=_addr(9) - 256), ALIAS), (dict(ws=_addr(6) - 256), ALIAS),
]


@pytest.mark.parametrize("over,want", BAD + [(dict(window=-1), CONTRACT), (dict(sink=-1), CONTRACT)])
def test_chunk_refuses(lib, over, want):
    assert _attend(lib, **over) == want


@pytest.mark.parametrize("over,want", BAD + [
    (dict(pcols=-1), SHAPE), (dict(pcols=1 << 31), SHAPE), (dict(pt=0), NULL), (dict(plen=0), NULL),
    (dict(pt=_addr(4) + 2), ALIGN), (dict(plen=_addr(5) + 1), ALIGN), (dict(out=_addr(4) - 32), ALIAS),
    (dict(lse=_addr(5)), ALIAS)])
def test_prefix_refuses(lib, over, want):
    assert _attend(lib, prefix=True, **over) == want


def test_workspace_grows_with_what_needs_it(lib):
    need = [_attend(lib, prefix, True) for prefix in (False, True)]
    assert 0 < need[0] < need[1] and all(n % 256 == 0 for n in need)
    for prefix, n in zip((False, True), need):
        # one byte less is refused; nothing in the size depends on addresses
        assert _attend(lib, prefix, wsb=n - 1) == WORKSPACE
        assert _attend(lib, prefix, True, k=_addr(30), v=_addr(31), bt=_addr(32)) == n
        assert _attend(lib, prefix, True, tokens=13) >= n
        for over in (dict(tokens=0), dict(tokens=-1), dict(hq=3), dict(reqs=0), dict(dim=96), dict(size=12)):
            assert _attend(lib, prefix, True, **over) == 0
        # any number of tokens and heads that a call may have
        assert _attend(lib, prefix, True, tokens=16777216, hq=126) > 0
        assert _attend(lib, prefix, True, tokens=30000, hq=65534) > 0


def test_attention_no_ops(lib):
    for prefix in (False, True):
        assert _attend(lib, prefix, tokens=0, q=0, out=0) == 0
        assert _attend(lib, prefix, reqs=0) == 0


def test_binding_refuses_host_tensors_and_shapes():
    q, c = torch.zeros(3, 4, 64), torch.zeros(2, 16, 2, 64)
    t, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    s = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(qsa.QSAError):
        qsa.qsa_qk_norm_rope(q, q, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(qsa.QSAError):
        qsa.qsa_chunk_attention(q, c, c, t, s, n)
    with pytest.raises(qsa.QSAError):
        qsa.qsa_prefix_attention(q, c, c, n, n, t, s, n)
