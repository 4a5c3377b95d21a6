"""Host-side checks of the paged-cache operators' C ABI and binding (no GPU):
every bad argument is refused before any CUDA call, so fake, never dereferenced
device addresses are enough."""
import ctypes
import os
import re

import pytest
import torch

import sparse_paged_attention_qsa_gb300 as qsa
from sparse_paged_attention_qsa_gb300 import binding
from sparse_paged_attention_qsa_gb300 import build as qbuild

HDR = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                   "qsa_cache.h")
NULL, DTYPE, SHAPE, STRIDE, ALIGN, CONTRACT, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 6, 7, 8


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load_library()


def _addr(k):
    return (1 << 36) * (k + 1)


FIELDS = ("k v pages size heads dim ks0 ks1 ks2 ks3 vs0 vs1 vs2 vs3 kscale vscale bt reqs cols bts0 "
          "dtype").split()


def _cache(over):
    a = dict(k=_addr(1), v=_addr(2), pages=64, size=16, heads=2, dim=64, ks0=2048, ks1=128, ks2=64,
             ks3=1, vs0=2048, vs1=128, vs2=64, vs3=1, kscale=0, vscale=0, bt=_addr(3), reqs=4,
             cols=8, bts0=8, dtype=1)
    for f in list(over):
        if f in a and f not in ("k_", "v_"):
            a[f] = over.pop(f)
    return binding._CACHE.pack(*[a[f] for f in FIELDS])


def _arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def test_header_constants_and_struct_match_the_binding():
    src = open(HDR).read()
    consts = dict(re.findall(r"#define\s+(QSA_\w+)\s+(\d+)u?\b", src))
    assert int(consts["QSA_DERR_CONTEXT"]) == qsa.DERR_CONTEXT == 32
    body = re.search(r"typedef struct qsa_paged_cache \{(.*?)\} qsa_paged_cache;", src, re.S)[1]
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    words = 0
    for decl in body.split(";"):
        for name in decl.split(","):
            n = re.search(r"\[(\d+)\]", name)
            words += int(n[1]) if n else bool(name.strip())
    assert words == len(FIELDS) == binding._CACHE.size // 8


def _append(lib, **over):
    cache = _cache(over)
    a = dict(cache=cache, nk=_addr(10), nv=_addr(11), dt=1, T=5, nks=_arr(128, 64, 1),
             nvs=_arr(128, 64, 1), t2r=_addr(12), ent=_addr(13), pos=_addr(14), ep=_addr(15),
             eps0=128, ws=_addr(16), wss0=128, ecols=128, err=_addr(17), stream=None)
    a.update(over)
    return lib.qsa_paged_append(*a.values())


def _attend(lib, **over):
    cache = _cache(over)
    a = dict(cache=cache, q=_addr(10), dt=1, n=1, hq=4, qs=_arr(256, 64, 1), ctx=_addr(11),
             scale=0.125, window=0, out=_addr(12), os=_arr(256, 64, 1), lse=_addr(13),
             win=_addr(14), ws0=128, wout=_addr(15), wos0=128, ecols=128, work=_addr(16), bytes=None,
             err=_addr(17), stream=None)
    a.update(over)
    if a["bytes"] is None:
        a["bytes"] = lib.qsa_paged_attention_workspace_bytes(cache, a["n"], a["hq"],
                                                             a["win"] is not None)
    return lib.qsa_paged_attention(*a.values())


def _evict(lib, **over):
    cache = _cache(over)
    a = dict(cache=cache, sums=_addr(10), ss0=128, pos=_addr(11), ps0=128, ecols=128, ctx=_addr(12),
             budget=32, sink=4, recent=8, kept=_addr(13), lens=_addr(14), so=_addr(15),
             po=_addr(16), err=_addr(18), stream=None)
    a.update(over)
    return lib.qsa_evict_entries(*a.values())


CACHE_REFUSALS = [
    (dict(dtype=3), DTYPE), (dict(dtype=0), DTYPE), (dict(kscale=_addr(30)), CONTRACT),
    (dict(vscale=_addr(30)), CONTRACT),
    (dict(dim=32), SHAPE), (dict(dim=96), SHAPE), (dict(dim=512), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=1025), SHAPE), (dict(size=4), SHAPE), (dict(size=24), SHAPE),
    (dict(size=131072), SHAPE), (dict(pages=-1), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(reqs=-1), SHAPE), (dict(reqs=65536), SHAPE), (dict(cols=-1), SHAPE),
    (dict(ks3=2), STRIDE), (dict(vs3=0), STRIDE), (dict(ks0=0), STRIDE), (dict(ks1=-128), STRIDE),
    (dict(ks2=65), STRIDE), (dict(vs1=132), STRIDE), (dict(vs0=1 << 39), STRIDE),
    (dict(ks1=64), STRIDE), (dict(ks0=1024), STRIDE), (dict(vs2=128), STRIDE),
    (dict(ks2=1024, ks1=64, ks0=1024), STRIDE), (dict(bts0=7), STRIDE), (dict(bts0=1 << 39), STRIDE),
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(bt=0), NULL),
    (dict(k=_addr(1) + 8), ALIGN), (dict(v=_addr(2) + 2), ALIGN), (dict(bt=_addr(3) + 2), ALIGN),
]


@pytest.mark.parametrize("call", [_append, _attend, _evict], ids=["append", "attend", "evict"])
@pytest.mark.parametrize("over,status", CACHE_REFUSALS)
def test_cache_descriptor_is_refused(lib, call, over, status):
    if call is _attend:
        over = dict(over, bytes=1 << 40)
    assert call(lib, **over) == status


@pytest.mark.parametrize("call", [_append, _attend, _evict], ids=["append", "attend", "evict"])
def test_no_descriptor(lib, call):
    assert call(lib, cache=None) == NULL


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), DTYPE), (dict(dt=2), DTYPE), (dict(dt=6), DTYPE), (dict(T=-1), SHAPE),
    (dict(T=(1 << 24) + 1), SHAPE), (dict(ecols=-1), SHAPE), (dict(ecols=1 << 31), SHAPE),
    (dict(nks=None), NULL), (dict(nvs=None), NULL), (dict(nk=None), NULL), (dict(nv=None), NULL),
    (dict(t2r=None), NULL), (dict(ent=None), NULL),
    (dict(nks=_arr(128, 64, 2)), STRIDE), (dict(nks=_arr(60, 64, 1)), STRIDE),
    (dict(nvs=_arr(128, 68, 1)), STRIDE), (dict(nvs=_arr(-128, 64, 1)), STRIDE),
    (dict(eps0=127), STRIDE), (dict(wss0=100), STRIDE),
    (dict(nk=_addr(10) + 2), ALIGN), (dict(ent=_addr(13) + 4), ALIGN), (dict(t2r=_addr(12) + 2), ALIGN),
    (dict(pos=_addr(14) + 4), ALIGN), (dict(ep=_addr(15) + 1), ALIGN), (dict(err=_addr(17) + 2), ALIGN),
    (dict(nk=_addr(1) + 64), ALIAS), (dict(t2r=_addr(2)), ALIAS), (dict(ep=_addr(1)), ALIAS),
    (dict(ws=_addr(13)), ALIAS), (dict(ep=_addr(16)), ALIAS), (dict(err=_addr(3)), ALIAS),
    (dict(bt=_addr(1) + 256), ALIAS),
])
def test_append_refusals(lib, over, status):
    assert _append(lib, **over) == status


def test_append_refuses_one_view_as_both(lib):
    assert _append(lib, v=_addr(1)) == ALIAS


def test_append_without_tokens_is_a_noop(lib):
    assert _append(lib, T=0, nk=None, nv=None, t2r=None, ent=None) == 0


@pytest.mark.parametrize("over,status", [
    (dict(dt=2), DTYPE), (dict(dt=6), DTYPE), (dict(scale=0.0), CONTRACT),
    (dict(scale=float("inf")), CONTRACT), (dict(scale=float("nan")), CONTRACT),
    (dict(scale=-1.0), CONTRACT), (dict(window=-1), CONTRACT),
    (dict(n=0), SHAPE), (dict(n=9), SHAPE), (dict(hq=3), SHAPE), (dict(hq=0), SHAPE),
    (dict(hq=65538), SHAPE), (dict(ecols=127), SHAPE), (dict(ecols=1 << 31), SHAPE),
    (dict(qs=None), NULL), (dict(os=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(ctx=None), NULL), (dict(win=None, bytes=1 << 40), NULL), (dict(wout=None), NULL),
    (dict(qs=_arr(256, 64, 2)), STRIDE), (dict(qs=_arr(0, 64, 1)), STRIDE),
    (dict(os=_arr(256, 4, 1)), STRIDE), (dict(os=_arr(64, 64, 1)), STRIDE),
    (dict(os=_arr(192, 64, 1)), STRIDE), (dict(ws0=127), STRIDE), (dict(wos0=1 << 39), STRIDE),
    (dict(q=_addr(10) + 8), ALIGN), (dict(out=_addr(12) + 8), ALIGN), (dict(ctx=_addr(11) + 2), ALIGN),
    (dict(lse=_addr(13) + 1), ALIGN), (dict(work=_addr(16) + 16), ALIGN), (dict(err=_addr(17) + 1), ALIGN),
    (dict(work=None), WORKSPACE), (dict(bytes=100), WORKSPACE),
    (dict(cols=4096, bts0=4096, win=None, wout=None, work=None), WORKSPACE),
    (dict(out=_addr(10)), ALIAS), (dict(out=_addr(1) + 4096), ALIAS), (dict(lse=_addr(12)), ALIAS),
    (dict(work=_addr(2)), ALIAS), (dict(wout=_addr(11)), ALIAS), (dict(err=_addr(12) + 4), ALIAS),
    (dict(wout=_addr(14) + 16), ALIAS), (dict(wout=_addr(14), wos0=129), ALIAS),
    (dict(out=_addr(14)), ALIAS),
])
def test_attention_refusals(lib, over, status):
    assert _attend(lib, **over) == status


@pytest.mark.parametrize("hq", [1 << 61, 1 << 62, (1 << 63) - 2])
def test_attention_head_counts_past_64_bits(lib, hq):
    # heads * next_n wraps to a small number for some of these
    assert _attend(lib, hq=hq, n=8, work=None, bytes=0) == SHAPE
    assert lib.qsa_paged_attention_workspace_bytes(_cache({}), 8, hq, 1) == 0


def test_attention_scales_past_binary32_are_refused(lib):
    most = 3.4028234e38
    assert _attend(lib, scale=most) == CONTRACT
    assert _attend(lib, scale=most / 1.5, q=None) == NULL      # that one is not


def test_attention_without_requests_is_a_noop(lib):
    assert _attend(lib, reqs=0, q=None, out=None, ctx=None, bytes=0, work=None) == 0


@pytest.mark.parametrize("over,status", [
    (dict(budget=0), CONTRACT), (dict(budget=(1 << 30) + 1), CONTRACT), (dict(sink=-1), CONTRACT),
    (dict(recent=-1), CONTRACT), (dict(sink=25), CONTRACT), (dict(sink=1 << 62), CONTRACT),
    (dict(ecols=-1), SHAPE), (dict(ecols=1 << 31, ss0=1 << 31, ps0=1 << 31), SHAPE),
    (dict(ss0=127), STRIDE), (dict(ps0=1), STRIDE),
    (dict(sums=None), NULL), (dict(pos=None), NULL), (dict(ctx=None), NULL), (dict(kept=None), NULL),
    (dict(lens=None), NULL), (dict(so=None), NULL), (dict(po=None), NULL),
    (dict(sums=_addr(10) + 2), ALIGN), (dict(kept=_addr(13) + 2), ALIGN), (dict(po=_addr(16) + 1), ALIGN),
    (dict(so=_addr(10)), ALIAS), (dict(po=_addr(11)), ALIAS), (dict(lens=_addr(12)), ALIAS),
    (dict(kept=_addr(15)), ALIAS), (dict(kept=_addr(1)), ALIAS), (dict(sums=_addr(2) + 64), ALIAS),
    (dict(so=_addr(1)), ALIAS), (dict(err=_addr(14)), ALIAS),
])
def test_evict_refusals(lib, over, status):
    assert _evict(lib, **over) == status


def _evict_strided(lib, **over):
    cache = _cache(over)
    a = dict(cache=cache, sums=_addr(10), ss0=128, pos=_addr(11), ps0=128, ecols=128, ctx=_addr(12),
             budget=32, sink=4, recent=8, kept=_addr(13), lens=_addr(14), so=_addr(15), so0=128,
             po=_addr(16), po0=128, err=_addr(18), stream=None)
    a.update(over)
    return lib.qsa_evict_entries_strided(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(so0=31), STRIDE), (dict(po0=0), STRIDE), (dict(so0=-128), STRIDE), (dict(po0=1 << 39), STRIDE),
    (dict(so=None), NULL), (dict(po=_addr(16) + 2), ALIGN), (dict(budget=0), CONTRACT),
    (dict(so=_addr(10)), ALIAS), (dict(po=_addr(11)), ALIAS),
    # between the other's rows: their extents overlap
    (dict(so=_addr(10) + 128), ALIAS), (dict(po=_addr(15) + 256), ALIAS),
    (dict(kept=_addr(15) + 3 * 512), ALIAS),
])
def test_evict_strided_refusals(lib, over, status):
    assert _evict_strided(lib, **over) == status


def test_evict_without_requests_is_a_noop(lib):
    assert _evict(lib, reqs=0) == 0


def test_workspace_queries(lib):
    w = lib.qsa_paged_attention_workspace_bytes
    short, long = _cache({}), _cache(dict(cols=4096, bts0=4096))
    assert w(short, 1, 8, 0) == 0                     # 128 entries: nothing is cut
    assert w(short, 1, 8, 1) >= 4 * 8 * (128 + 1) * 4
    assert w(long, 1, 8, 0) > 0
    assert w(long, 1, 8, 1) >= w(long, 1, 8, 0) + 4 * 8 * 65536 * 4
    for n, hq in ((0, 8), (9, 8), (1, 7), (1, 0), (2, 65536)):
        assert w(long, n, hq, 0) == 0
    assert w(None, 1, 8, 0) == 0 and w(_cache(dict(reqs=0, cols=4096, bts0=4096)), 1, 8, 1) == 0
    # logits past any address space: refused
    huge = dict(reqs=65535, cols=1 << 26, bts0=1 << 26)
    assert w(_cache(dict(huge)), 8, 8192, 1) == 0


def test_short_tables_need_no_workspace(lib):
    # refused for another reason, or launched (which fails here): never for the workspace
    assert _attend(lib, win=None, wout=None, work=None, bytes=0, q=None) == NULL


def test_binding_refuses_host_tensors():
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    bt, i32 = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    f = torch.zeros((1, 64))
    for call in (lambda: qsa.qsa_paged_append(k[0, :1], k[0, :1], k, k, bt, i32, i32.long()),
                 lambda: qsa.qsa_paged_attention(k[0, :1], k, k, bt, i32),
                 lambda: qsa.qsa_evict_entries(f, bt, i32, k, k, bt, 8)):
        with pytest.raises(qsa.QSAError):
            call()


class _Recorder:
    """Stands in for the library: says what it would have been given."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096

        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    """The binding on host tensors in front of a recorder: nothing can be launched."""
    rec = _Recorder()
    monkeypatch.setattr(binding, "_lib", rec)
    monkeypatch.setattr(binding, "load_library", lambda: rec)
    monkeypatch.setattr(binding, "_on_current_device", lambda *t: None)
    monkeypatch.setattr(binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    monkeypatch.setattr(binding, "_launch_stream", lambda s, d: 0)
    return rec


def _workspace_calls(ws):
    h = dict(dtype=torch.float16)
    i32, i64 = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    bt = torch.zeros((1, 1), dtype=torch.int32)
    kv = torch.zeros((1, 512, 2, 256), **h)
    sel = (torch.zeros((1, 4, 128), **h), torch.zeros((1, 128, 1, 128), **h), bt, i32, i32, i64)
    att = (torch.zeros((1, 3, 256), **h), kv[:, :, :1], kv[:, :, 1:], bt)
    return [lambda: qsa.qsa_select_paged_tokens(*sel, workspace=ws),
            lambda: qsa.qsa_sparse_attention(*att, i32, torch.zeros((1, 2051), dtype=torch.int32),
                                             workspace=ws),
            lambda: qsa.qsa_select_attend(*sel, *att, workspace=ws),
            lambda: qsa.qsa_paged_attention(*att, i32, workspace=ws)]


@pytest.mark.parametrize("which", range(4))
def test_a_workspace_that_holds_less_than_its_elements_is_refused(recorder, which):
    one = torch.zeros(1, dtype=torch.uint8)
    wide = torch.zeros(200, dtype=torch.uint8)
    for ws in (one.expand(1 << 20), wide.as_strided((100, 100), (1, 1)), wide[::2]):
        with pytest.raises(qsa.QSAError) as e:
            _workspace_calls(ws)[which]()
        assert e.value.status == WORKSPACE
    assert not recorder.calls
    _workspace_calls(wide)[which]()                  # one that is what it says goes on
    (name, args), = recorder.calls
    assert args[args.index(wide.data_ptr()) + 1] == 200, name


def test_evict_outputs_wider_than_the_budget(recorder):
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    bt, lens = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    sums, pos = torch.zeros((2, 32)), torch.zeros((2, 32), dtype=torch.int32)

    def call(so, po):
        return qsa.qsa_evict_entries(sums, pos, lens, k, k, bt, 24, weight_sums_out=so,
                                     entry_positions_out=po)

    so, po = torch.zeros((2, 40)), torch.zeros((2, 32), dtype=torch.int32)
    assert call(so, po)[2:] == (so, po)
    call(so[:, :24], po[:, 8:])
    call(torch.zeros((2, 24)), torch.zeros(48, dtype=torch.int32))
    got = [(a[12], a[13], a[14], a[15]) for _, a in recorder.calls]
    assert got[0] == (so.data_ptr(), 40, po.data_ptr(), 32)
    assert got[1] == (so.data_ptr(), 40, po.data_ptr() + 32, 32)
    assert (got[2][1], got[2][3]) == (24, 24)
    recorder.calls.clear()
    for bad, status in ((torch.zeros((2, 23)), SHAPE), (torch.zeros((3, 24)), SHAPE),
                        (torch.zeros(96), SHAPE), (torch.zeros((2, 32), dtype=torch.float64), DTYPE),
                        (torch.zeros((32, 2)).t(), STRIDE)):
        with pytest.raises(qsa.QSAError) as e:
            call(bad, po)
        assert e.value.status == status
    assert not recorder.calls


@pytest.mark.parametrize("budget", [0, -1, (1 << 30) + 1, 1 << 60, 1 << 70])
def test_evict_budgets_are_refused_before_results_are_allocated(recorder, budget):
    assert binding._MAX_ENTRIES == int(re.search(r"QSA_CACHE_MAX_ENTRIES (\d+)", open(HDR).read())[1])
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    bt, lens = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_evict_entries(torch.zeros((2, 32)), bt.repeat(1, 16), lens, k, k, bt, budget)
    assert e.value.status == CONTRACT and not recorder.calls
