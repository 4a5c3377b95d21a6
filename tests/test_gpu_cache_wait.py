"""Failure detection in the dense paged attention: a device wait that runs out.

As test_gpu_wait_timeout.py, through libqsa_waittest.so (stage waits of 2 ms
and a symbol that leaves one slot fill of the walk's first CTA without a
copy): the call returns with the timeout bit set, whether its runs are joined
by a second kernel or within a cluster, and the next call on the same stream
and workspace is right again, as is the product library in the same context.
No trap, no bad address and no endless loop is involved."""
import ctypes
import time

import pytest
import torch

import sparse_paged_attention_qsa_gb300 as qsa
from sparse_paged_attention_qsa_gb300 import build as qbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("lens,fill", [([60000, 3, 9000], 3), ([60000, 3, 9000], 0), ([3000, 800], 2),
                                       ([40] * 20, 1)],
                         ids=["joined", "first", "cluster", "whole"])
@pytest.mark.parametrize("cache", [torch.float16, torch.float8_e4m3fn])
def test_attention_wait_runs_out_then_next_call_is_exact(lens, fill, cache):
    lib = ctypes.CDLL(qbuild.build_wait_test())
    qsa.declare_signatures(lib)
    lib.qsa_test_withhold_paged_fill.restype = None
    lib.qsa_test_withhold_paged_fill.argtypes = [ctypes.c_int32]
    gen = torch.Generator(device=DEV).manual_seed(5)
    cols = -(-max(lens) // 64)
    shape = (len(lens) * cols, 64, 2, 64)
    k, v = (torch.randn(shape, generator=gen, device=DEV).to(cache) for _ in range(2))
    tables = torch.arange(len(lens) * cols, dtype=torch.int32, device=DEV).view(len(lens), cols)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn((len(lens), 6, 64), generator=gen, device=DEV).half()
    sums = torch.zeros((len(lens), cols * 64), device=DEV)
    ws = torch.empty(qsa.qsa_paged_attention_workspace_bytes(k, v, tables, num_heads=6,
                                                             with_weights=True),
                     dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(library=None):
        added = torch.zeros_like(sums)
        out = qsa.qsa_paged_attention(q, k, v, tables, ctx, weight_sums=sums,
                                      weight_sums_out=added, workspace=ws, error_word=err,
                                      library=library)
        torch.cuda.synchronize()
        return out, added

    ref = call()
    assert int(err.item()) == 0
    lib.qsa_test_withhold_paged_fill(-1)
    assert all(torch.equal(a, b) for a, b in zip(call(lib), ref))     # the test build, healthy
    assert int(err.item()) == 0
    try:
        lib.qsa_test_withhold_paged_fill(fill)
        t0 = time.perf_counter()
        call(lib)
        dt = time.perf_counter() - t0
    finally:
        lib.qsa_test_withhold_paged_fill(-1)
    assert int(err.item()) & qsa.DERR_TIMEOUT, int(err.item())
    assert dt < 5.0, dt
    err.zero_()
    for library in (lib, None):
        assert all(torch.equal(a, b) for a, b in zip(call(library), ref))
    assert int(err.item()) == 0
