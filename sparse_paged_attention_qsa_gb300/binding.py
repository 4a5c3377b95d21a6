"""Thin ctypes binding over libqsa (include/qsa.h).

Argument marshalling only: tensors become (data pointer, dtype tag, shape,
strides); the stream is torch's current CUDA stream unless given.  Every step
of the computation runs in libqsa's CUDA kernels.  PyTorch is used here for
device memory (outputs and workspaces the caller did not pass) and streams.

If libqsa.so has not been built the first call raises -- there is no
fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqsa.so")

TOKEN_TOPK = 2048
COMPRESS_RATIO = 4
TOPK_BLOCKS = 512
OUT_WIDTH = 2051
DERR_REQUEST, DERR_CMP_PAGE, DERR_KV_PAGE, DERR_TIMEOUT = 1, 2, 4, 8
DERR_IDX_BLOCK = 16
DERR_CONTEXT = 32
IDX_HEAD_DIM, IDX_MAX_TOPK = 128, 2048

DT_F16, DT_BF16, DT_F32, DT_I32, DT_I64, DT_F8E4M3 = 1, 2, 3, 4, 5, 6
_DTYPE_TAG = {torch.float16: DT_F16, torch.bfloat16: DT_BF16, torch.float32: DT_F32,
              torch.int32: DT_I32, torch.int64: DT_I64, torch.float8_e4m3fn: DT_F8E4M3}

STATUS = {0: "QSA_OK", 1: "QSA_ERR_NULL", 2: "QSA_ERR_DTYPE", 3: "QSA_ERR_SHAPE",
          4: "QSA_ERR_STRIDE", 5: "QSA_ERR_ALIGN", 6: "QSA_ERR_CONTRACT",
          7: "QSA_ERR_WORKSPACE", 8: "QSA_ERR_ALIAS", 9: "QSA_ERR_CUDA",
          10: "QSA_ERR_SCRATCH_LIMIT"}

EXPORTED = ("qsa_status_string", "qsa_version", "qsa_select_workspace_bytes",
            "qsa_select_paged_tokens", "qsa_attention_workspace_bytes",
            "qsa_sparse_attention", "qsa_select_attend_workspace_bytes", "qsa_select_attend",
            "qsa_select_attend_fused_rows",
            "qsa_select_attend_fused_cluster",
            "qsa_static_scratch_bytes",
            "qsa_select_paged_tokens_static_scratch", "qsa_build_metadata",
            "qsa_paged_mqa_logits", "qsa_top_k_per_row_decode",
            "qsa_paged_append", "qsa_paged_attention_workspace_bytes", "qsa_paged_attention",
            "qsa_evict_entries", "qsa_evict_entries_strided")


class QSAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


_lock = threading.Lock()
_lib = None


def load_library(path: str | None = None):
    """Load libqsa.so (once) and declare the C signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"libqsa.so not found at {path}; build it with "
                "`python -m sparse_paged_attention_qsa_gb300.build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(path)
        declare_signatures(lib)
        _lib = lib
        return lib


class _Only:
    """Attribute access on a library that may lack some entry points (a
    test build carries a subset): missing ones are skipped."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        try:
            return getattr(self._lib, name)
        except AttributeError:
            return _Sink()


class _Sink:
    def __setattr__(self, name, value):
        pass


def declare_signatures(lib):
    """Declare the C signatures of include/*.h on a loaded library handle."""
    full = lib
    lib = _Only(full)
    i32, i64, u64, vp, sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                             ctypes.c_void_p, ctypes.c_size_t)
    p64 = ctypes.POINTER(ctypes.c_int64)
    lib.qsa_status_string.restype = ctypes.c_char_p
    lib.qsa_status_string.argtypes = [ctypes.c_int]
    lib.qsa_version.restype = ctypes.c_int
    lib.qsa_version.argtypes = []
    lib.qsa_select_workspace_bytes.restype = sz
    lib.qsa_select_workspace_bytes.argtypes = [i64, i64]
    lib.qsa_attention_workspace_bytes.restype = sz
    lib.qsa_attention_workspace_bytes.argtypes = [i64, i64]
    lib.qsa_select_paged_tokens.restype = ctypes.c_int
    lib.qsa_select_paged_tokens.argtypes = [
        vp, ctypes.c_int, i64, p64,
        vp, ctypes.c_int, p64, p64,
        vp, ctypes.c_int, i64, i64, i64,
        vp, ctypes.c_int, vp, ctypes.c_int, vp, ctypes.c_int,
        i32, i32,
        vp, ctypes.c_int, i64, i64,
        vp, sz, vp, vp]
    lib.qsa_static_scratch_bytes.restype = sz
    lib.qsa_static_scratch_bytes.argtypes = []
    lib.qsa_select_paged_tokens_static_scratch.restype = ctypes.c_int
    lib.qsa_select_paged_tokens_static_scratch.argtypes = [
        vp, ctypes.c_int, i64, p64,
        vp, ctypes.c_int, p64, p64,
        vp, ctypes.c_int, i64, i64, i64,
        vp, ctypes.c_int, vp, ctypes.c_int, vp, ctypes.c_int,
        i32, i32,
        vp, ctypes.c_int, i64, i64,
        vp, vp]
    lib.qsa_sparse_attention.restype = ctypes.c_int
    lib.qsa_sparse_attention.argtypes = [
        vp, ctypes.c_int, i64, p64,
        vp, vp, ctypes.c_int, p64, p64, p64,
        vp, ctypes.c_int, i64, i64, i64,
        vp, ctypes.c_int,
        vp, ctypes.c_int, i64, i64,
        ctypes.c_float,
        vp, ctypes.c_int, p64,
        vp, sz, vp, vp]
    lib.qsa_select_attend_fused_rows.restype = i64
    lib.qsa_select_attend_fused_rows.argtypes = [ctypes.c_int]
    lib.qsa_select_attend_fused_cluster.restype = i64
    lib.qsa_select_attend_fused_cluster.argtypes = [i64, i64, ctypes.c_int]
    lib.qsa_select_attend_workspace_bytes.restype = sz
    lib.qsa_select_attend_workspace_bytes.argtypes = [i64, i64]
    lib.qsa_select_attend.restype = ctypes.c_int
    lib.qsa_select_attend.argtypes = [
        vp, ctypes.c_int, i64, p64,
        vp, ctypes.c_int, p64, p64,
        vp, ctypes.c_int, i64, i64, i64,
        vp, ctypes.c_int, vp, ctypes.c_int, vp, ctypes.c_int,
        i32, i32,
        vp, ctypes.c_int, i64, i64,
        vp, ctypes.c_int, p64,
        vp, vp, ctypes.c_int, p64, p64, p64,
        vp, ctypes.c_int, i64, i64,
        ctypes.c_float,
        vp, ctypes.c_int, p64,
        vp, sz, vp, vp]
    lib.qsa_build_metadata.restype = ctypes.c_int
    lib.qsa_build_metadata.argtypes = [
        vp, ctypes.c_int, vp, ctypes.c_int, vp, ctypes.c_int,
        vp, ctypes.c_int, i64, i64, i64, i64,
        i64, i64, i64, i64, i64, i64,
        vp, vp, vp, vp, vp, i64, vp]
    lib.qsa_paged_mqa_logits.restype = ctypes.c_int
    lib.qsa_paged_mqa_logits.argtypes = [
        vp, ctypes.c_int, i64, i64,
        vp, ctypes.c_int, i64, i64,
        vp, ctypes.c_int,
        vp, ctypes.c_int, i64,
        vp, ctypes.c_int, i64, i64,
        i64,
        vp, ctypes.c_int, i64, i64,
        vp, vp]
    lib.qsa_top_k_per_row_decode.restype = ctypes.c_int
    lib.qsa_top_k_per_row_decode.argtypes = [
        vp, ctypes.c_int, i64, i64, i64, i64, i64,
        vp, ctypes.c_int, i64,
        i64, vp, ctypes.c_int, i64, vp]
    lib.qsa_paged_append.restype = ctypes.c_int
    lib.qsa_paged_append.argtypes = [
        vp, vp, vp, ctypes.c_int, i64, vp, vp, vp, vp, vp, vp, i64, vp, i64, i64, vp, vp]
    lib.qsa_paged_attention_workspace_bytes.restype = sz
    lib.qsa_paged_attention_workspace_bytes.argtypes = [vp, i64, i64, ctypes.c_int]
    lib.qsa_paged_attention.restype = ctypes.c_int
    lib.qsa_paged_attention.argtypes = [
        vp, vp, ctypes.c_int, i64, i64, vp, vp, ctypes.c_float, i64,
        vp, vp, vp, vp, i64, vp, i64, i64, vp, sz, vp, vp]
    lib.qsa_evict_entries.restype = ctypes.c_int
    lib.qsa_evict_entries.argtypes = [
        vp, vp, i64, vp, i64, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.qsa_evict_entries_strided.restype = ctypes.c_int
    lib.qsa_evict_entries_strided.argtypes = [
        vp, vp, i64, vp, i64, i64, vp, i64, i64, i64, vp, vp, vp, i64, vp, i64, vp, vp]
    return full


def _arr(vals):
    vals = list(vals)
    return (ctypes.c_int64 * len(vals))(*vals)


def _tag(t: torch.Tensor) -> int:
    return _DTYPE_TAG.get(t.dtype, 0)


def _ptr(t: torch.Tensor | None) -> int | None:
    # the library reads and writes device memory only: a host tensor's address
    # would reach a kernel as an invalid device address
    if t is None:
        return None
    if t.device.type != "cuda":
        raise QSAError(1, f"every tensor must be in CUDA device memory (got a {t.device} tensor)")
    return t.data_ptr() or None


def _on_current_device(*tensors):
    """Every tensor given must be in the memory of the current CUDA device,
    which the library runs on: a host tensor, or one on another GPU, would
    reach a kernel as an invalid address."""
    cur = None
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()                  # -1: host memory
        if d < 0:
            raise QSAError(1, f"every tensor must be in CUDA device memory (got a {t.device} "
                              "tensor)")
        if cur is None:
            cur = torch.cuda.current_device()
        if d != cur:
            raise QSAError(1, f"a tensor is on cuda:{d} but the current device is cuda:{cur} "
                              "(select it with torch.cuda.device)")


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int):
    if status != 0:
        raise QSAError(status, load_library().qsa_status_string(status).decode())


def qsa_select_workspace_bytes(num_rows: int, cmp_pt_cols: int) -> int:
    return int(load_library().qsa_select_workspace_bytes(num_rows, cmp_pt_cols))


def qsa_attention_workspace_bytes(num_rows: int, index_width: int) -> int:
    return int(load_library().qsa_attention_workspace_bytes(num_rows, index_width))


def _workspace(nbytes: int, device) -> torch.Tensor:
    # torch's CUDA allocator returns 512-byte aligned blocks
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _workspace_bytes(workspace) -> int:
    """What the library may write behind a caller's workspace."""
    if not workspace.is_contiguous():      # a broadcast or strided one holds less than numel says
        raise QSAError(7, "workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def qsa_select_paged_tokens(q_sel, cmp_cache, cmp_page_table, token_to_request, seq_lens,
                            query_positions, token_topk: int = TOKEN_TOPK,
                            compress_ratio: int = COMPRESS_RATIO, out=None, workspace=None,
                            error_word=None, stream=None, library=None):
    """Selection: returns out [R,2051] int32 (see include/qsa.h).  `library`:
    another loaded build of the C ABI (declare_signatures) instead of libqsa."""
    lib = library or load_library()
    _on_current_device(q_sel, cmp_cache, cmp_page_table, token_to_request, seq_lens,
                       query_positions, out, workspace, error_word)
    R = q_sel.shape[0] if q_sel.dim() == 3 else -1
    if q_sel.dim() != 3 or cmp_cache.dim() != 4 or cmp_page_table.dim() != 2:
        raise QSAError(3, "q_sel must be [R,4,128], cmp_cache [P,128,1,128], page table 2-D")
    if tuple(q_sel.shape[1:]) != (4, 128):
        raise QSAError(3, "q_sel must be [R,4,128]")
    if out is None:
        out = torch.empty((R, OUT_WIDTH), dtype=torch.int32, device=q_sel.device)
    if cmp_page_table.stride(1) != 1 and cmp_page_table.shape[1] > 1:
        raise QSAError(4, "page table columns must be contiguous")
    if out.dim() != 2 or (out.stride(1) != 1 and out.shape[1] > 1):
        raise QSAError(4, "out must be [R,2051] with contiguous columns")
    cols = cmp_page_table.shape[1]
    need = qsa_select_workspace_bytes(R, cols)
    if workspace is None:
        workspace = _workspace(need, q_sel.device)
    st = lib.qsa_select_paged_tokens(
        _ptr(q_sel), _tag(q_sel), R, _arr(q_sel.stride()),
        _ptr(cmp_cache), _tag(cmp_cache), _arr(cmp_cache.shape), _arr(cmp_cache.stride()),
        _ptr(cmp_page_table), _tag(cmp_page_table), cmp_page_table.shape[0], cols,
        cmp_page_table.stride(0),
        _ptr(token_to_request), _tag(token_to_request), _ptr(seq_lens), _tag(seq_lens),
        _ptr(query_positions), _tag(query_positions),
        int(token_topk), int(compress_ratio),
        _ptr(out), _tag(out), out.shape[1], out.stride(0),
        _ptr(workspace), _workspace_bytes(workspace),
        _ptr(error_word), _stream(stream))
    _check(st)
    return out


def qsa_sparse_attention(q, k_cache, v_cache, kv_page_table, token_to_request, indices,
                         scale: float = 1.0 / 16.0, out=None, workspace=None, error_word=None,
                         stream=None):
    """Sparse attention: returns out [R,3,256] FP16 (see include/qsa.h).
    k_cache / v_cache are the exact-packed views (strides [262144,512,256,1],
    V at storage offset 256 of the same buffer)."""
    lib = load_library()
    _on_current_device(q, k_cache, v_cache, kv_page_table, token_to_request, indices, out,
                       workspace, error_word)
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.dim() != 4 or indices.dim() != 2:
        raise QSAError(3, "q [R,3,256], k/v [P,512,1,256], indices [R,W] expected")
    if k_cache.shape != v_cache.shape:
        raise QSAError(3, "k_cache and v_cache shapes differ")
    R = q.shape[0]
    if out is None:
        out = torch.empty((R, 3, 256), dtype=torch.float16, device=q.device)
    if kv_page_table.dim() != 2 or (kv_page_table.stride(1) != 1 and kv_page_table.shape[1] > 1):
        raise QSAError(4, "page table must be 2-D with contiguous columns")
    if indices.stride(1) != 1 and indices.shape[1] > 1:
        raise QSAError(4, "index columns must be contiguous")
    width = indices.shape[1]
    need = qsa_attention_workspace_bytes(R, width)
    if workspace is None:
        workspace = _workspace(need, q.device)
    st = lib.qsa_sparse_attention(
        _ptr(q), _tag(q), R, _arr(q.stride()),
        _ptr(k_cache), _ptr(v_cache), _tag(k_cache) if k_cache.dtype == v_cache.dtype else 0,
        _arr(k_cache.shape), _arr(k_cache.stride()), _arr(v_cache.stride()),
        _ptr(kv_page_table), _tag(kv_page_table), kv_page_table.shape[0], kv_page_table.shape[1],
        kv_page_table.stride(0),
        _ptr(token_to_request), _tag(token_to_request),
        _ptr(indices), _tag(indices), width, indices.stride(0),
        float(scale),
        _ptr(out), _tag(out), _arr(out.stride()),
        _ptr(workspace), _workspace_bytes(workspace),
        _ptr(error_word), _stream(stream))
    _check(st)
    return out


def qsa_decode(q_sel, cmp_cache, cmp_page_table, token_to_request, seq_lens, query_positions,
               q_attn, k_cache, v_cache, kv_page_table, scale: float = 1.0 / 16.0,
               indices=None, out=None, sel_workspace=None, att_workspace=None,
               error_word=None, stream=None):
    """One decode step of the whole path: selection then sparse attention on
    the same stream (the index list stays on the device)."""
    indices = qsa_select_paged_tokens(q_sel, cmp_cache, cmp_page_table, token_to_request,
                                      seq_lens, query_positions, out=indices,
                                      workspace=sel_workspace, error_word=error_word,
                                      stream=stream)
    out = qsa_sparse_attention(q_attn, k_cache, v_cache, kv_page_table, token_to_request,
                               indices, scale=scale, out=out, workspace=att_workspace,
                               error_word=error_word, stream=stream)
    return indices, out


def qsa_select_attend_workspace_bytes(num_rows: int, cmp_pt_cols: int) -> int:
    return int(load_library().qsa_select_attend_workspace_bytes(num_rows, cmp_pt_cols))


def qsa_select_attend_fused_rows(cmp_dtype=torch.float16) -> int:
    """The largest batch qsa_select_attend runs as one fused kernel on the
    current device (include/qsa.h)."""
    return int(load_library().qsa_select_attend_fused_rows(_DTYPE_TAG.get(cmp_dtype, 0)))


def qsa_select_attend_fused_cluster(num_rows: int, cmp_pt_cols: int,
                                    cmp_dtype=torch.float16) -> int:
    """CTAs per row's cluster with which qsa_select_attend runs this batch
    as one fused kernel on the current device, 0 = the chained kernels
    (include/qsa.h)."""
    return int(load_library().qsa_select_attend_fused_cluster(
        num_rows, cmp_pt_cols, _DTYPE_TAG.get(cmp_dtype, 0)))


def qsa_select_attend(q_sel, cmp_cache, cmp_page_table, token_to_request, seq_lens,
                      query_positions, q_attn, k_cache, v_cache, kv_page_table,
                      scale: float = 1.0 / 16.0, indices=None, out=None, workspace=None,
                      error_word=None, stream=None, library=None):
    """One decode step in one call (include/qsa.h, qsa_select_attend): the
    selection's indices [R,2051] int32 and the attention output [R,3,256]
    FP16.  Both page tables are indexed by token_to_request.  `library` as in
    qsa_select_paged_tokens."""
    lib = library or load_library()
    _on_current_device(q_sel, cmp_cache, cmp_page_table, token_to_request, seq_lens,
                       query_positions, q_attn, k_cache, v_cache, kv_page_table, indices, out,
                       workspace, error_word)
    if q_sel.dim() != 3 or cmp_cache.dim() != 4 or cmp_page_table.dim() != 2:
        raise QSAError(3, "q_sel must be [R,4,128], cmp_cache [P,128,1,128], page table 2-D")
    if q_attn.dim() != 3 or k_cache.dim() != 4 or v_cache.dim() != 4 or kv_page_table.dim() != 2:
        raise QSAError(3, "q_attn [R,3,256], k/v [P,512,1,256], K/V page table 2-D expected")
    if k_cache.shape != v_cache.shape:
        raise QSAError(3, "k_cache and v_cache shapes differ")
    if kv_page_table.shape[0] != cmp_page_table.shape[0]:
        raise QSAError(3, "both page tables need one row per request")
    for t in (cmp_page_table, kv_page_table):
        if t.stride(1) != 1 and t.shape[1] > 1:
            raise QSAError(4, "page table columns must be contiguous")
    R = q_sel.shape[0]
    if indices is None:
        indices = torch.empty((R, OUT_WIDTH), dtype=torch.int32, device=q_sel.device)
    if indices.dim() != 2 or (indices.stride(1) != 1 and indices.shape[1] > 1):
        raise QSAError(4, "indices must be [R,2051] with contiguous columns")
    if out is None:
        out = torch.empty((R, 3, 256), dtype=torch.float16, device=q_sel.device)
    cols = cmp_page_table.shape[1]
    need = qsa_select_attend_workspace_bytes(R, cols)
    if workspace is None:
        workspace = _workspace(need, q_sel.device)
    st = lib.qsa_select_attend(
        _ptr(q_sel), _tag(q_sel), R, _arr(q_sel.stride()),
        _ptr(cmp_cache), _tag(cmp_cache), _arr(cmp_cache.shape), _arr(cmp_cache.stride()),
        _ptr(cmp_page_table), _tag(cmp_page_table), cmp_page_table.shape[0], cols,
        cmp_page_table.stride(0),
        _ptr(token_to_request), _tag(token_to_request), _ptr(seq_lens), _tag(seq_lens),
        _ptr(query_positions), _tag(query_positions),
        TOKEN_TOPK, COMPRESS_RATIO,
        _ptr(indices), _tag(indices), indices.shape[1], indices.stride(0),
        _ptr(q_attn), _tag(q_attn), _arr(q_attn.stride()),
        _ptr(k_cache), _ptr(v_cache), _tag(k_cache) if k_cache.dtype == v_cache.dtype else 0,
        _arr(k_cache.shape), _arr(k_cache.stride()), _arr(v_cache.stride()),
        _ptr(kv_page_table), _tag(kv_page_table), kv_page_table.shape[1],
        kv_page_table.stride(0),
        float(scale),
        _ptr(out), _tag(out), _arr(out.stride()),
        _ptr(workspace), _workspace_bytes(workspace),
        _ptr(error_word), _stream(stream))
    _check(st)
    return indices, out


def qsa_build_metadata(query_start_loc, seq_lens, block_table, num_tokens: int, *,
                       storage_block_size: int, compress_ratio: int,
                       circular_buffer_size: int = 0, common_slot_mapping=None,
                       num_mapped_tokens: int | None = None, max_num_work: int = 0,
                       out=None, stream=None):
    """Side-cache metadata (include/qsa_metadata.h).  Returns a dict of
    device tensors: token_to_req int32, logical_positions int64,
    visible_blocks int32, slot_mapping int64 (each [num_tokens]) and, when
    max_num_work > 0, work_metadata int32 [max_num_work, 2].

    ``num_mapped_tokens`` is the host's copy of query_start_loc[-1]; when it
    is not given it is read from the device (one synchronising read).
    ``out`` may hold preallocated tensors under the same keys."""
    lib = load_library()
    _on_current_device(query_start_loc, seq_lens, block_table, common_slot_mapping,
                       *(out or {}).values())
    dev = query_start_loc.device
    num_reqs = query_start_loc.numel() - 1
    if query_start_loc.dim() != 1 or seq_lens.dim() != 1 or block_table.dim() != 2:
        raise QSAError(3, "query_start_loc and seq_lens 1-D, block_table 2-D expected")
    if not query_start_loc.is_contiguous() or not seq_lens.is_contiguous():
        raise QSAError(4, "query_start_loc and seq_lens must be contiguous")
    if seq_lens.numel() < num_reqs:
        raise QSAError(3, "seq_lens shorter than the request count")
    if num_mapped_tokens is None:
        num_mapped_tokens = int(query_start_loc[-1].item())
    out = dict(out or {})
    T = int(num_tokens)
    for key, dt in (("token_to_req", torch.int32), ("logical_positions", torch.int64),
                    ("visible_blocks", torch.int32), ("slot_mapping", torch.int64)):
        if key not in out:
            out[key] = torch.empty(T, dtype=dt, device=dev)
    if max_num_work and "work_metadata" not in out:
        out["work_metadata"] = torch.empty((max_num_work, 2), dtype=torch.int32, device=dev)
    work = out.get("work_metadata")
    for key in ("token_to_req", "logical_positions", "visible_blocks", "slot_mapping"):
        if out[key].numel() < T or not out[key].is_contiguous():
            raise QSAError(3, f"{key} must be a contiguous tensor of >= num_tokens entries")
    if work is not None and (not work.is_contiguous() or work.numel() < 2 * max_num_work):
        raise QSAError(3, "work_metadata must be contiguous [max_num_work, 2]")
    common = common_slot_mapping
    st = lib.qsa_build_metadata(
        _ptr(query_start_loc), _tag(query_start_loc), _ptr(seq_lens), _tag(seq_lens),
        _ptr(common), _tag(common) if common is not None else 0,
        _ptr(block_table), _tag(block_table), block_table.shape[0], block_table.shape[1],
        block_table.stride(0), block_table.stride(1),
        num_reqs, int(num_mapped_tokens), T,
        int(storage_block_size), int(compress_ratio), int(circular_buffer_size),
        _ptr(out["token_to_req"]), _ptr(out["logical_positions"]),
        _ptr(out["visible_blocks"]), _ptr(out["slot_mapping"]),
        _ptr(work) if max_num_work else None, int(max_num_work), _stream(stream))
    _check(st)
    return out


def qsa_paged_mqa_logits(q, kv_cache, weights, context_lens, block_tables, next_n: int,
                         max_model_len: int, *, block_size: int, out=None, error_word=None,
                         stream=None, library=None):
    """Weighted paged MQA indexer logits (include/qsa_indexer.h): returns fp32
    [rows, max_model_len].  q is E4M3 [rows, heads, 128]; kv_cache holds
    [num_blocks, block_size*132] bytes (uint8 or float8_e4m3fn storage).
    `library` as in qsa_select_paged_tokens."""
    lib = library or load_library()
    _on_current_device(q, kv_cache, weights, context_lens, block_tables, out, error_word)
    if q.dim() != 3 or kv_cache.dim() != 2 or weights.dim() != 2 or block_tables.dim() != 2:
        raise QSAError(3, "q [rows,H,128], kv_cache [blocks, bs*132], weights [rows,H], "
                          "block_tables 2-D expected")
    if not (q.is_contiguous() and kv_cache.is_contiguous() and weights.is_contiguous()
            and context_lens.is_contiguous()):
        raise QSAError(4, "q, kv_cache, weights and context_lens must be contiguous")
    if kv_cache.shape[1] != block_size * (IDX_HEAD_DIM + 4):
        raise QSAError(3, "kv_cache rows must hold block_size * 132 bytes")
    if block_tables.shape[1] > 1 and block_tables.stride(1) != 1:
        raise QSAError(4, "block-table columns must be contiguous")
    rows, heads = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((rows, max_model_len), dtype=torch.float32, device=q.device)
    if out.dim() != 2 or (out.shape[1] > 1 and out.stride(1) != 1):
        raise QSAError(4, "logits must be 2-D with contiguous columns")
    kv_tag = DT_F8E4M3 if kv_cache.dtype in (torch.uint8, torch.float8_e4m3fn) else 0
    st = lib.qsa_paged_mqa_logits(
        _ptr(q), _tag(q), rows, heads,
        _ptr(kv_cache), kv_tag, kv_cache.shape[0], int(block_size),
        _ptr(weights), _tag(weights),
        _ptr(context_lens), _tag(context_lens), context_lens.numel(),
        _ptr(block_tables), _tag(block_tables), block_tables.shape[1], block_tables.stride(0),
        int(next_n),
        _ptr(out), _tag(out), int(max_model_len), out.stride(0),
        _ptr(error_word), _stream(stream))
    _check(st)
    return out


def qsa_top_k_per_row_decode(logits, next_n: int, seq_lens, topk_tokens: int, out=None,
                             stream=None):
    """Per-row top-k of the indexer logits (include/qsa_indexer.h): returns
    int32 [rows, topk_tokens], -1 padded."""
    lib = load_library()
    _on_current_device(logits, seq_lens, out)
    if logits.dim() != 2:
        raise QSAError(3, "logits must be 2-D")
    rows, cols = logits.shape
    if out is None:
        out = torch.empty((rows, topk_tokens), dtype=torch.int32, device=logits.device)
    if out.dim() != 2 or (out.shape[1] > 1 and out.stride(1) != 1):
        raise QSAError(4, "indices must be 2-D with contiguous columns")
    st = lib.qsa_top_k_per_row_decode(
        _ptr(logits), _tag(logits), rows, cols, logits.stride(0), logits.stride(1),
        int(next_n), _ptr(seq_lens), _tag(seq_lens), seq_lens.numel(),
        int(topk_tokens), _ptr(out), _tag(out), out.stride(0), _stream(stream))
    _check(st)
    return out


# --- the paged K/V cache operators (include/qsa_cache.h) ------------------------

_CACHE = struct.Struct("21q")       # qsa_paged_cache: 8-byte fields throughout
_STRIDES3 = struct.Struct("3q")
_MAX_ENTRIES = 1 << 30              # QSA_CACHE_MAX_ENTRIES


def _cache_struct(k_cache, v_cache, block_tables, k_scale, v_scale) -> bytes:
    """A qsa_paged_cache of K and V views [pages, page_size, heads, dim].  Types
    that the C struct does not carry are checked here."""
    if k_cache.dim() != 4 or v_cache.dim() != 4 or block_tables.dim() != 2:
        raise QSAError(3, "k/v caches [pages, page_size, heads, dim] and a 2-D block table expected")
    shape = k_cache.shape
    if shape != v_cache.shape:
        raise QSAError(3, "k_cache and v_cache shapes differ")
    if k_cache.dtype != v_cache.dtype:
        raise QSAError(2, "k_cache and v_cache dtypes differ")
    if block_tables.dtype != torch.int32:
        raise QSAError(2, "block_tables must be int32")
    reqs, cols = block_tables.shape
    s0, s1 = block_tables.stride()
    if s1 != 1 and cols > 1:
        raise QSAError(4, "block-table columns must be contiguous")
    ks = vs = 0
    if k_scale is not None:
        ks = _scale_ptr(k_scale, shape[2])
    if v_scale is not None:
        vs = _scale_ptr(v_scale, shape[2])
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), *shape, *k_cache.stride(),
                       *v_cache.stride(), ks, vs, block_tables.data_ptr(), reqs, cols,
                       s0 if reqs > 1 else max(s0, cols), _DTYPE_TAG.get(k_cache.dtype, 0))


def _scale_ptr(scale, heads) -> int:
    if scale.dtype != torch.float32:
        raise QSAError(2, "K/V scales must be float32")
    if scale.dim() != 1 or scale.shape[0] != heads or not scale.is_contiguous():
        raise QSAError(3, "K/V scales must be contiguous [heads]")
    return scale.data_ptr()


def _typed(t, dtype, dims, what) -> int:
    """The address of an argument whose C type is fixed (0 for None)."""
    if t is None:
        return 0
    if t.dtype != dtype:
        raise QSAError(2, f"{what} must be {dtype}")
    if t.dim() != dims:
        raise QSAError(3, f"{what} must be {dims}-D")
    return t.data_ptr()


def _flat(t, dtype, n, what) -> int:
    """As _typed, for a contiguous tensor of exactly n elements."""
    if t is None:
        return 0
    if t.dtype != dtype:
        raise QSAError(2, f"{what} must be {dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise QSAError(3, f"{what} must be contiguous, {n} elements")
    return t.data_ptr()


def _rows(t, dtype, reqs, what):
    """(address, row stride) of a [reqs, cols] per-entry array."""
    if t is None:
        return 0, 0
    p = _typed(t, dtype, 2, what)
    n, cols = t.shape
    s0, s1 = t.stride()
    if n != reqs:
        raise QSAError(3, f"{what} needs one row per request")
    if s1 != 1 and cols > 1:
        raise QSAError(4, f"{what} columns must be contiguous")
    return p, s0 if reqs > 1 else max(s0, cols)


def _budget_rows(t, dtype, reqs, budget, what):
    """(address, row stride) of an output of `budget` columns a request: contiguous
    with that many elements, or the first columns of a wider [reqs, cols] array."""
    if t.dtype == dtype and t.numel() == reqs * budget and t.is_contiguous():
        return t.data_ptr(), budget
    p, s0 = _rows(t, dtype, reqs, what)
    if t.shape[1] < budget:
        raise QSAError(3, f"{what} must hold {budget} columns")
    return p, s0


def _word(t) -> int:
    return _flat(t, torch.int32, 1, "error_word")


def _launch_stream(stream, device_index) -> int:
    # the current stream's handle without building a Stream object around it
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device_index)
    return _stream(stream) or 0


def _on_stream(stream, device_index):
    """A context in which torch allocates for the launch stream, so that a
    buffer made here is not handed out again while the launch uses it."""
    if stream is None:
        return _HERE
    raw = _stream(stream) or 0
    if raw == torch._C._cuda_getCurrentRawStream(device_index):
        return _HERE
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                             else torch.cuda.ExternalStream(raw))


_HERE = contextlib.nullcontext()
_raw_alloc = torch._C._cuda_cudaCachingAllocator_raw_alloc if torch.version.cuda else None
_raw_free = torch._C._cuda_cudaCachingAllocator_raw_delete if torch.version.cuda else None


def _need_tensor(t, what):
    if not isinstance(t, torch.Tensor):
        raise QSAError(1, f"{what} must be a tensor")


def qsa_paged_append(k, v, k_cache, v_cache, block_tables, token_to_request, entries, *,
                     k_scale=None, v_scale=None, positions=None, entry_positions=None,
                     weight_sums=None, error_word=None, stream=None):
    """Write new tokens' keys and values [T, heads, dim] into a paged cache
    (include/qsa_cache.h): token t becomes entry entries[t] (int64, -1 =
    padding) of request token_to_request[t] (int32).  entry_positions (int32)
    and weight_sums (fp32), [requests, entries], get the token's position and
    0.  Returns (k_cache, v_cache)."""
    lib = _lib or load_library()
    _on_current_device(k, v, k_cache, v_cache, block_tables, token_to_request, entries, k_scale,
                       v_scale, positions, entry_positions, weight_sums, error_word)
    if k.dim() != 3 or k.shape != v.shape or k.shape[1:] != k_cache.shape[2:]:
        raise QSAError(3, "k and v must be [tokens, heads, dim] of the cache's heads and dim")
    if k.dtype != v.dtype:
        raise QSAError(2, "k and v dtypes differ")
    T = k.shape[0]
    cache = _cache_struct(k_cache, v_cache, block_tables, k_scale, v_scale)
    reqs = block_tables.shape[0]
    pos, pos_s0 = _rows(entry_positions, torch.int32, reqs, "entry_positions")
    sums, sums_s0 = _rows(weight_sums, torch.float32, reqs, "weight_sums")
    cols = [t.shape[1] for t in (entry_positions, weight_sums) if t is not None]
    _check(lib.qsa_paged_append(
        cache, k.data_ptr(), v.data_ptr(), _tag(k), T, _STRIDES3.pack(*k.stride()),
        _STRIDES3.pack(*v.stride()), _flat(token_to_request, torch.int32, T, "token_to_request"),
        _flat(entries, torch.int64, T, "entries"), _flat(positions, torch.int64, T, "positions"),
        pos, pos_s0, sums, sums_s0, min(cols) if cols else 0, _word(error_word),
        _launch_stream(stream, k.get_device())))
    return k_cache, v_cache


def qsa_paged_attention_workspace_bytes(k_cache, v_cache, block_tables, *, next_n: int = 1,
                                        num_heads: int, with_weights: bool = False) -> int:
    """Bytes of workspace that qsa_paged_attention needs for this cache."""
    return int(load_library().qsa_paged_attention_workspace_bytes(
        _cache_struct(k_cache, v_cache, block_tables, None, None), next_n, num_heads,
        bool(with_weights)))


def qsa_paged_attention(q, k_cache, v_cache, block_tables, context_lens, *, next_n: int = 1,
                        scale: float | None = None, window: int = 0, k_scale=None, v_scale=None,
                        out=None, lse=None, weight_sums=None, weight_sums_out=None,
                        workspace=None, error_word=None, stream=None, library=None):
    """Dense attention of each request's next_n new tokens, q [requests*next_n,
    heads, dim], over its cached entries (include/qsa_cache.h).  scale: 1/sqrt
    (dim) unless given.  lse: fp32 [rows, heads], filled when given.
    weight_sums / weight_sums_out: fp32 [requests, entries]; the second gets
    the first plus the weight that each entry received in this call.  Returns
    out [rows, heads, dim].  `library` as in qsa_select_paged_tokens."""
    lib = library or _lib or load_library()
    _on_current_device(q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale, out,
                       lse, weight_sums, weight_sums_out, workspace, error_word)
    if q.dim() != 3:
        raise QSAError(3, "q must be [requests * next_n, heads, dim]")
    cache = _cache_struct(k_cache, v_cache, block_tables, k_scale, v_scale)
    rows, heads, dim = q.shape
    reqs = block_tables.shape[0]
    if rows != reqs * next_n or dim != k_cache.shape[3]:
        raise QSAError(3, "q must be [requests * next_n, heads, dim] of the cache's dim")
    device = q.get_device()
    raw = _launch_stream(stream, device)
    weights = weight_sums is not None or weight_sums_out is not None
    need = lib.qsa_paged_attention_workspace_bytes(cache, next_n, heads, weights) \
        if workspace is None else 0
    if out is None:
        if stream is None:
            out = torch.empty((rows, heads, dim), dtype=q.dtype, device=q.device)
        else:
            with _on_stream(stream, device):
                out = torch.empty((rows, heads, dim), dtype=q.dtype, device=q.device)
    if out.dtype != q.dtype:
        raise QSAError(2, "out must have q's dtype")
    if out.shape != q.shape:
        raise QSAError(3, "out must have q's shape")
    sums, sums_s0 = _rows(weight_sums, torch.float32, reqs, "weight_sums")
    souts, souts_s0 = _rows(weight_sums_out, torch.float32, reqs, "weight_sums_out")
    entry_cols = min([t.shape[1] for t in (weight_sums, weight_sums_out) if t is not None]) \
        if weights else 0
    ctx = _flat(context_lens, torch.int32, reqs, "context_lens")
    lse_ptr, word = _flat(lse, torch.float32, rows * heads, "lse"), _word(error_word)
    if workspace is None:
        # from torch's allocator, for the launch stream, without a tensor around it
        # (which costs the host 2 to 3 us more, as much as a launch)
        ws = _raw_alloc(need, raw) if need else 0
    else:
        ws, need = workspace.data_ptr(), _workspace_bytes(workspace)
    try:
        status = lib.qsa_paged_attention(
            cache, q.data_ptr(), _tag(q), next_n, heads, _STRIDES3.pack(*q.stride()), ctx,
            dim ** -0.5 if scale is None else scale, window, out.data_ptr(),
            _STRIDES3.pack(*out.stride()), lse_ptr, sums, sums_s0, souts, souts_s0, entry_cols,
            ws, need, word, raw)
    finally:
        if workspace is None and ws:
            _raw_free(ws)        # back to the stream's pool: what comes next on it follows the launch
    _check(status)
    return out


def qsa_evict_entries(weight_sums, entry_positions, context_lens, k_cache, v_cache, block_tables,
                      budget: int, *, num_sink: int = 0, num_recent: int = 0, kept=None,
                      new_lens=None, weight_sums_out=None, entry_positions_out=None,
                      error_word=None, stream=None):
    """Cut every request down to at most `budget` cached entries, keeping the
    first num_sink positions, the num_recent newest and then those of the
    largest weight_sums; K and V are moved within the cache
    (include/qsa_cache.h).  Returns (kept int32 [requests, budget], new_lens
    int32 [requests], weight_sums_out fp32, entry_positions_out int32
    [requests, budget]).  weight_sums_out and entry_positions_out may be given
    wider, as the next step's append and attention need them: their columns
    from budget on stay as they are."""
    lib = _lib or load_library()
    _on_current_device(weight_sums, entry_positions, context_lens, k_cache, v_cache, block_tables,
                       kept, new_lens, weight_sums_out, entry_positions_out, error_word)
    cache = _cache_struct(k_cache, v_cache, block_tables, None, None)
    reqs = block_tables.shape[0]
    sums, sums_s0 = _rows(weight_sums, torch.float32, reqs, "weight_sums")
    pos, pos_s0 = _rows(entry_positions, torch.int32, reqs, "entry_positions")
    if not sums or not pos:
        for t, what in ((weight_sums, "weight_sums"), (entry_positions, "entry_positions")):
            _need_tensor(t, what)
    device, dev = block_tables.get_device(), block_tables.device
    raw = _launch_stream(stream, device)
    if not 1 <= budget <= _MAX_ENTRIES:    # before anything of that size is allocated
        raise QSAError(6, f"budget must be 1 to {_MAX_ENTRIES}")
    if kept is None or new_lens is None or weight_sums_out is None or entry_positions_out is None:
        with _on_stream(stream, device):
            if kept is None:
                kept = torch.empty((reqs, budget), dtype=torch.int32, device=dev)
            if new_lens is None:
                new_lens = torch.empty(reqs, dtype=torch.int32, device=dev)
            if weight_sums_out is None:
                weight_sums_out = torch.empty((reqs, budget), dtype=torch.float32, device=dev)
            if entry_positions_out is None:
                entry_positions_out = torch.empty((reqs, budget), dtype=torch.int32, device=dev)
    souts, souts_s0 = _budget_rows(weight_sums_out, torch.float32, reqs, budget, "weight_sums_out")
    pouts, pouts_s0 = _budget_rows(entry_positions_out, torch.int32, reqs, budget,
                                   "entry_positions_out")
    _check(lib.qsa_evict_entries_strided(
        cache, sums, sums_s0, pos, pos_s0,
        min(weight_sums.shape[1], entry_positions.shape[1]),
        _flat(context_lens, torch.int32, reqs, "context_lens"), budget, num_sink, num_recent,
        _flat(kept, torch.int32, reqs * budget, "kept"),
        _flat(new_lens, torch.int32, reqs, "new_lens"), souts, souts_s0, pouts, pouts_s0,
        _word(error_word), raw))
    return kept, new_lens, weight_sums_out, entry_positions_out
