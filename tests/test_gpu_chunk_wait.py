"""Failure detection in the chunk attention: a device wait that runs out.

As test_gpu_cache_wait.py, through libqsa_waittest.so (waits of 2 ms and a symbol
that leaves one slot fill of the walk's first CTA without a copy, K's and V's
tiles counted in turn): the call returns with the timeout bit set, and the next
call on the same stream and workspace is right again, as is the product library
in the same context.  No trap, no bad address and no endless loop is involved.
(The batches give the first CTA, one of 152, more tiles than the fill's number.)"""
import ctypes
import time

import pytest
import torch

import sparse_paged_attention_qsa_gb300 as qsa
from sparse_paged_attention_qsa_gb300 import build as qbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("reqs,prefix,fill", [
    ([(1, 200000), (2, 0), (1, 5000)], None, 0), ([(1, 200000), (2, 0), (1, 5000)], None, 3),
    ([(4000, 900), (2000, 0)], None, 2), ([(4000, 900), (2000, 0)], None, 9), ([(1, 20)] * 400, 8000, 1),
    ([(90, 60)] * 150, None, 5)],
    ids=["first K", "long V", "prompt K", "prompt V", "prefix", "edges"])
@pytest.mark.parametrize("cache", [torch.float16, torch.float8_e4m3fn])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_wait_runs_out_then_next_call_is_exact(reqs, prefix, fill, cache, dtype):
    if cache == torch.float16 and dtype == torch.bfloat16:
        cache = dtype
    lib = ctypes.CDLL(qbuild.build_wait_test())
    qsa.declare_signatures(lib)
    lib.qsa_test_withhold_chunk_fill.restype = None
    lib.qsa_test_withhold_chunk_fill.argtypes = [ctypes.c_int32]
    gen = torch.Generator(device=DEV).manual_seed(5)
    lens = [n + old for n, old in reqs]
    cols, pcols = -(-max(lens) // 64), -(-(prefix or 0) // 64)
    shape = (len(lens) * cols + pcols, 64, 2, 64)
    k, v = (torch.randn(shape, generator=gen, device=DEV).to(cache) for _ in range(2))
    ids = torch.arange(shape[0], dtype=torch.int32, device=DEV)
    tables, ptable = ids[pcols:].view(len(lens), cols), ids[:pcols]
    plen = torch.tensor([prefix or 0], dtype=torch.int32, device=DEV)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0] + [n for n, _ in reqs], device=DEV).cumsum(0).to(torch.int32)
    q = torch.randn((int(starts[-1]), 8, 64), generator=gen, device=DEV).to(dtype)
    ws = torch.empty(qsa.qsa_chunk_attention_workspace_bytes(
        k, v, tables, num_tokens=q.shape[0], num_heads=8, prefix_cols=pcols if prefix else -1),
        dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(library=None):
        lse = torch.zeros(q.shape[:2], device=DEV)
        kw = dict(workspace=ws, error_word=err, library=library, lse=lse)
        if prefix:
            out = qsa.qsa_prefix_attention(q, k, v, ptable, plen, tables, starts, ctx, **kw)
        else:
            out = qsa.qsa_chunk_attention(q, k, v, tables, starts, ctx, **kw)
        torch.cuda.synchronize()
        return out, lse

    ref = call()
    assert int(err.item()) == 0
    lib.qsa_test_withhold_chunk_fill(-1)
    assert all(torch.equal(a, b) for a, b in zip(call(lib), ref))     # the test build, healthy
    assert int(err.item()) == 0
    try:
        lib.qsa_test_withhold_chunk_fill(fill)
        t0 = time.perf_counter()
        call(lib)
        assert time.perf_counter() - t0 < 20
        assert int(err.item()) & qsa.DERR_TIMEOUT
    finally:
        lib.qsa_test_withhold_chunk_fill(-1)
    err.zero_()
    for library in (lib, None):
        assert all(torch.equal(a, b) for a, b in zip(call(library), ref))
        assert int(err.item()) == 0
