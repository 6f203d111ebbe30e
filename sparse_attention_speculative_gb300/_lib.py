"""ctypes binding of libvsd (include/vsd.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch supplies device memory and the current stream.  If libvsd.so is
missing the calls raise immediately; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvsd.so")

_lock = threading.Lock()
_lib = None

VSD_OK = 0
STATUS_NAMES = {
    -1: "VSD_ERR_INVALID_ARG",
    -2: "VSD_ERR_UNSUPPORTED",
    -3: "VSD_ERR_CUDA",
    -4: "VSD_ERR_WORKSPACE",
    -5: "VSD_ERR_TIMEOUT",
}
DEV_BAD_BLOCK = 0x1
DEV_BAD_INDEX = 0x2
DEV_BAD_LENGTH = 0x4
DEV_TIMEOUT = 0x8
STEP_RECORD_ROWS = 0x1
STEP_REUSE_ROWS = 0x2
STEP_EARLY_GATHER = 0x4
SPARSE_VERIFY_EARLY_GATHER = 0x4
VERIFY_EARLY_PREFETCH = 0x4


class VsdError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = "%s failed: %s" % (what, STATUS_NAMES.get(status, str(status)))
        if status == -3 and _lib is not None:
            msg += " (cudaError %d)" % _lib.vsd_last_cuda_error()
        super().__init__(msg)


class Geom(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_blocks_per_seq", ctypes.c_int), ("num_blocks", ctypes.c_int)]


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libvsd.so (built by ``sparse_attention_speculative_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError("libvsd.so is not built (%s); run "
                               "`python -m sparse_attention_speculative_gb300.build`" % path)
        lib = ctypes.CDLL(path)
        P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        GP = ctypes.POINTER(Geom)
        lib.vsd_verify_workspace_size.argtypes = [GP, I, I, ctypes.POINTER(SZ)]
        lib.vsd_verify_attn_collect.argtypes = [GP, I, P, P, P, P, P, I, I, I, F, P, P, P, P, SZ, P]
        lib.vsd_verify_attn_collect_noalloc.argtypes = [GP, I, P, P, P, P, P, I, I, I, F, P, P,
                                                        P, P]
        lib.vsd_verify_attn_collect_all.argtypes = [GP, I, P, P, P, P, P, I, F, P, P, P, P, SZ,
                                                    P]
        lib.vsd_sparse_verify_workspace_size.argtypes = [GP, I, I, ctypes.POINTER(SZ)]
        lib.vsd_sparse_verify_attn.argtypes = [GP, I, P, P, P, P, P, P, P, I, ctypes.c_uint, F, P,
                                                P, SZ, P]
        lib.vsd_verify_attn_collect_srh.argtypes = [GP, I, P, P, P, P, P, I, I, P, I, F, P, P, P,
                                                    P, SZ, P]
        lib.vsd_select_hybrid_workspace_size.argtypes = [I, I, ctypes.POINTER(SZ)]
        lib.vsd_select_topk_hybrid.argtypes = [I, I, P, I, P, P, I, I, I, I, I, P, P, P, SZ, P]
        lib.vsd_select_workspace_size.argtypes = [I, I, I, I, ctypes.POINTER(SZ)]
        lib.vsd_select_topk.argtypes = [I, I, P, P, I, I, I, I, P, P, P, P, SZ, P]
        lib.vsd_sparse_workspace_size.argtypes = [GP, I, I, ctypes.POINTER(SZ)]
        lib.vsd_sparse_decode_attn.argtypes = [GP, P, P, P, P, P, P, I, P, P, I, F, P, P, SZ, P]
        lib.vsd_verify_attn_collect_scored.argtypes = [GP, I, P, P, P, P, P, I, I, I, F, P, P,
                                                       P, P, I, I, ctypes.c_uint, P, P, P, P, SZ,
                                                       P]
        lib.vsd_select_topk_scored.argtypes = [I, P, P, P, I, I, I, I, P, P, P]
        lib.vsd_page_key_means.argtypes = [GP, P, P, P, P, I, P, P]
        lib.vsd_copy.argtypes = [P, P, SZ, P]
        lib.vsd_append_kv.argtypes = [GP, I, P, P, P, P, I, P, P, P]
        lib.vsd_sparse_decode_attn_step.argtypes = [GP, P, P, P, P, P, P, P, P, I, P, P, I, P,
                                                    ctypes.c_uint, F, P, P, SZ, P]
        lib.vsd_advance_lengths.argtypes = [I, I, P, I, P, P, P, I, P, P]
        lib.vsd_append_kv_quant.argtypes = [P, I, P, P, P, P, I, P, P, P, P, P, P]
        lib.vsd_read_kv_quant.argtypes = [P, I, P, P, P, P, P, P, I, P, P, P, P]
        lib.vsd_verify_quant_workspace_size.argtypes = [P, I, I, ctypes.POINTER(SZ)]
        lib.vsd_verify_attn_collect_quant.argtypes = [P, I, P, P, P, P, P, P, P, I, I, I, F, P,
                                                      P, P, P, I, I, P, P, SZ, P]
        lib.vsd_sparse_quant_workspace_size.argtypes = [P, I, I, ctypes.POINTER(SZ)]
        lib.vsd_sparse_decode_attn_quant.argtypes = [P, P, P, P, P, P, P, P, P, I, P, P, I, F, P,
                                                     P, SZ, P]
        lib.vsd_block_topk.argtypes = [GP, I, P, P, P, I, I, F, P, P, P]
        lib.vsd_read_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint)]
        lib.vsd_get_error_string.argtypes = [I]
        lib.vsd_get_error_string.restype = ctypes.c_char_p
        lib.vsd_last_cuda_error.argtypes = []
        for name in ("vsd_verify_workspace_size", "vsd_verify_attn_collect",
                     "vsd_verify_attn_collect_all", "vsd_sparse_verify_workspace_size",
                     "vsd_verify_attn_collect_srh", "vsd_select_hybrid_workspace_size",
                     "vsd_select_topk_hybrid",
                     "vsd_sparse_verify_attn",
                     "vsd_verify_attn_collect_noalloc",
                     "vsd_select_workspace_size", "vsd_select_topk", "vsd_sparse_workspace_size",
                     "vsd_sparse_decode_attn", "vsd_page_key_means", "vsd_block_topk",
                     "vsd_verify_attn_collect_scored", "vsd_select_topk_scored", "vsd_copy",
                     "vsd_append_kv_quant", "vsd_read_kv_quant", "vsd_verify_quant_workspace_size",
                     "vsd_verify_attn_collect_quant", "vsd_sparse_quant_workspace_size",
                     "vsd_sparse_decode_attn_quant",
                     "vsd_append_kv", "vsd_advance_lengths", "vsd_sparse_decode_attn_step",
                     "vsd_read_device_status", "vsd_last_cuda_error"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _check(rc: int, what: str) -> None:
    if rc != VSD_OK:
        raise VsdError(rc, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def geom_for(B: int, Hq: int, k_cache: torch.Tensor, block_table: torch.Tensor) -> Geom:
    NB, Hkv, page, d = k_cache.shape
    return Geom(B, Hq, Hkv, d, page, int(block_table.shape[1]), NB)


_ws_cache = {}


def _workspace(nbytes: int, device, tag: str) -> Optional[torch.Tensor]:
    """Cached device scratch, one buffer per (call kind, device, size), zero-filled
    when allocated as the workspace contract asks (every call leaves it reusable by
    calls of the same kind; the kinds whose counters are laid out per (sequence, KV
    head) carry B * Hkv in their tag)."""
    if nbytes == 0:
        return None
    key = (tag, str(device), nbytes)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = torch.zeros(nbytes + 256, dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    off = (-ws.data_ptr()) % 256
    return ws[off:off + nbytes]


def vsd_verify_workspace_size(geom: Geom, R: int, P_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().vsd_verify_workspace_size(ctypes.byref(geom), R, P_max, ctypes.byref(out)),
           "vsd_verify_workspace_size")
    return int(out.value)


def vsd_verify_attn_collect(q, k_cache, v_cache, block_table, prefix_len, *, P_max: int,
                            scale: float, row0: int = 0, row1: Optional[int] = None,
                            logits=None, partial=None, out=None, collect: bool = True,
                            workspace=None, stream=None):
    """Verification attention + Collect-2-Query.  Returns (out, logits, partial)."""
    lib = load()
    B, R, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(block_table, torch.int32, "block_table")
    _need(prefix_len, torch.int32, "prefix_len")
    geom = geom_for(B, Hq, k_cache, block_table)
    if row1 is None:
        row1 = R - 1
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if collect:
        if logits is None:
            logits = torch.empty((B, 2, Hq, P_max), dtype=torch.float32, device=dev)
        if partial is None:
            partial = torch.empty((B, geom.Hkv, P_max), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(vsd_verify_workspace_size(geom, R, P_max), dev, "verify")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.vsd_verify_attn_collect(ctypes.byref(geom), R, _ptr(q), _ptr(k_cache),
                                     _ptr(v_cache), _ptr(block_table), _ptr(prefix_len),
                                     int(row0), int(row1), int(P_max), float(scale),
                                     _ptr(logits), _ptr(partial), _ptr(out), _ptr(workspace),
                                     ws_bytes, _stream(stream))
    _check(rc, "vsd_verify_attn_collect")
    return out, logits, partial


def vsd_verify_attn_collect_all(q, k_cache, v_cache, block_table, prefix_len, *, P_max: int,
                                scale: float, logits=None, partial=None, out=None,
                                collect: bool = True, workspace=None, stream=None):
    """Verification collecting every verify row (logits fp32 [B, R, Hq, P_max]; the
    partial scores sum all R rows).  Returns (out, logits, partial)."""
    lib = load()
    B, R, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(block_table, torch.int32, "block_table")
    _need(prefix_len, torch.int32, "prefix_len")
    geom = geom_for(B, Hq, k_cache, block_table)
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if collect:
        if logits is None:
            logits = torch.empty((B, R, Hq, P_max), dtype=torch.float32, device=dev)
        if partial is None:
            partial = torch.empty((B, geom.Hkv, P_max), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(vsd_verify_workspace_size(geom, R, P_max), dev, "verify")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.vsd_verify_attn_collect_all(ctypes.byref(geom), R, _ptr(q), _ptr(k_cache),
                                         _ptr(v_cache), _ptr(block_table), _ptr(prefix_len),
                                         int(P_max), float(scale), _ptr(logits), _ptr(partial),
                                         _ptr(out), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "vsd_verify_attn_collect_all")
    return out, logits, partial


def vsd_verify_attn_collect_noalloc(q, k_cache, v_cache, block_table, prefix_len, *,
                                    P_max: int, scale: float, row0: int = 0,
                                    row1: Optional[int] = None, logits=None, partial=None,
                                    out=None, collect: bool = True, stream=None):
    """vsd_verify_attn_collect with the library's fixed device scratch instead of a
    workspace (the C call allocates nothing; outputs are allocated here when not
    given).  Returns (out, logits, partial)."""
    lib = load()
    B, R, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(block_table, torch.int32, "block_table")
    _need(prefix_len, torch.int32, "prefix_len")
    geom = geom_for(B, Hq, k_cache, block_table)
    if row1 is None:
        row1 = R - 1
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if collect:
        if logits is None:
            logits = torch.empty((B, 2, Hq, P_max), dtype=torch.float32, device=dev)
        if partial is None:
            partial = torch.empty((B, geom.Hkv, P_max), dtype=torch.float32, device=dev)
    rc = lib.vsd_verify_attn_collect_noalloc(ctypes.byref(geom), R, _ptr(q), _ptr(k_cache),
                                             _ptr(v_cache), _ptr(block_table),
                                             _ptr(prefix_len), int(row0), int(row1),
                                             int(P_max), float(scale), _ptr(logits),
                                             _ptr(partial), _ptr(out), _stream(stream))
    _check(rc, "vsd_verify_attn_collect_noalloc")
    return out, logits, partial


def vsd_select_topk(partial, prefix_len, *, k: int, n_sink: int, n_recent: int, idx=None,
                    n_sel=None, scores_out=None, want_scores: bool = False,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Protected top-k over the aggregated score.  partial: fp32 [n_rows, Hkv, P_max]."""
    lib = load()
    _need(partial, torch.float32, "partial")
    _need(prefix_len, torch.int32, "prefix_len")
    n_rows, Hkv, P_max = partial.shape
    dev = partial.device
    if idx is None:
        idx = torch.empty((n_rows, k), dtype=torch.int32, device=dev)
    if n_sel is None:
        n_sel = torch.empty((n_rows,), dtype=torch.int32, device=dev)
    if want_scores and scores_out is None:
        scores_out = torch.empty((n_rows, P_max), dtype=torch.float32, device=dev)
    rc = lib.vsd_select_topk(n_rows, Hkv, _ptr(partial), _ptr(prefix_len), P_max, int(k),
                             int(n_sink), int(n_recent), _ptr(idx), _ptr(n_sel),
                             _ptr(scores_out), None, 0, _stream(stream))
    _check(rc, "vsd_select_topk")
    return idx, n_sel, scores_out


def vsd_sparse_workspace_size(geom: Geom, k_max: int, max_tail: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().vsd_sparse_workspace_size(ctypes.byref(geom), int(k_max), int(max_tail),
                                            ctypes.byref(out)), "vsd_sparse_workspace_size")
    return int(out.value)


def vsd_sparse_decode_attn(q, k_cache, v_cache, block_table, idx, n_sel, tail_start, seq_len,
                           *, scale: float, max_tail: int, out=None, workspace=None,
                           stream=None):
    """Sparse draft-step attention.  q: bf16 [B, Hq, d]; idx: int32 [B, k_max] or None."""
    lib = load()
    B, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    _need(tail_start, torch.int32, "tail_start")
    _need(seq_len, torch.int32, "seq_len")
    geom = geom_for(B, Hq, k_cache, block_table)
    k_max = 0 if idx is None else int(idx.shape[1])
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = _workspace(vsd_sparse_workspace_size(geom, k_max, max_tail), q.device,
                               "sparse:%d" % (geom.B * geom.Hkv))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.vsd_sparse_decode_attn(ctypes.byref(geom), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_table), _ptr(idx), _ptr(n_sel), k_max,
                                    _ptr(tail_start), _ptr(seq_len), int(max_tail), float(scale),
                                    _ptr(out), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "vsd_sparse_decode_attn")
    return out


def vsd_read_device_status(stream=None) -> int:
    flags = ctypes.c_uint(0)
    _check(load().vsd_read_device_status(_stream(stream), ctypes.byref(flags)),
           "vsd_read_device_status")
    return int(flags.value)


def vsd_sparse_verify_workspace_size(geom: Geom, R: int, k_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().vsd_sparse_verify_workspace_size(ctypes.byref(geom), int(R), int(k_max),
                                                   ctypes.byref(out)),
           "vsd_sparse_verify_workspace_size")
    return int(out.value)


def vsd_sparse_verify_attn(q, k_cache, v_cache, block_table, prefix_len, idx, n_sel, *,
                           scale: float, flags: int = 0, out=None, workspace=None, stream=None):
    """Sparse verification: verify row t attends idx[b, :n_sel[b]] and the verify block
    positions P_b .. P_b + t.  q: bf16 [B, R, Hq, d]; idx: int32 [B, k_max].  flags: 0 or
    SPARSE_VERIFY_EARLY_GATHER.  Returns out."""
    lib = load()
    B, R, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    _need(prefix_len, torch.int32, "prefix_len")
    _need(idx, torch.int32, "idx")
    _need(n_sel, torch.int32, "n_sel")
    geom = geom_for(B, Hq, k_cache, block_table)
    k_max = int(idx.shape[1])
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = _workspace(vsd_sparse_verify_workspace_size(geom, R, k_max), q.device,
                               "sparse_verify")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.vsd_sparse_verify_attn(ctypes.byref(geom), R, _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_table), _ptr(prefix_len), _ptr(idx), _ptr(n_sel),
                                    k_max, int(flags), float(scale), _ptr(out), _ptr(workspace),
                                    ws_bytes, _stream(stream))
    _check(rc, "vsd_sparse_verify_attn")
    return out


def vsd_verify_attn_collect_srh(q, k_cache, v_cache, block_table, prefix_len, head_mask, *,
                                P_max: int, scale: float, row0: int = 0,
                                row1: Optional[int] = None, logits=None, partial=None,
                                out=None, workspace=None, stream=None):
    """Verification with the collected logits and partial scores restricted to the query
    heads with head_mask[h] != 0 (uint8 [Hq] on the device).  Returns (out, logits,
    partial); the logits of the other heads are left untouched."""
    lib = load()
    B, R, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    _need(head_mask, torch.uint8, "head_mask")
    geom = geom_for(B, Hq, k_cache, block_table)
    if row1 is None:
        row1 = R - 1
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if logits is None:
        logits = torch.zeros((B, 2, Hq, P_max), dtype=torch.float32, device=dev)
    if partial is None:
        partial = torch.empty((B, geom.Hkv, P_max), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(vsd_verify_workspace_size(geom, R, P_max), dev, "verify")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.vsd_verify_attn_collect_srh(ctypes.byref(geom), R, _ptr(q), _ptr(k_cache),
                                         _ptr(v_cache), _ptr(block_table), _ptr(prefix_len),
                                         int(row0), int(row1), _ptr(head_mask), int(P_max),
                                         float(scale), _ptr(logits), _ptr(partial), _ptr(out),
                                         _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "vsd_verify_attn_collect_srh")
    return out, logits, partial


def vsd_select_topk_hybrid(partial_target, partial_draft, prefix_len, *, k: int, m: int,
                           n_sink: int, n_recent: int, idx=None, n_sel=None, workspace=None,
                           stream=None):
    """Dustin's hybrid budget: protected sinks and recent window, then the top-m by the
    draft score, then the rest by the target score.  partial_*: fp32 [n_rows, Hkv*, P_max]."""
    lib = load()
    _need(partial_target, torch.float32, "partial_target")
    _need(partial_draft, torch.float32, "partial_draft")
    _need(prefix_len, torch.int32, "prefix_len")
    n_rows, Hkv_t, P_max = partial_target.shape
    Hkv_d = int(partial_draft.shape[1])
    assert partial_draft.shape[0] == n_rows and partial_draft.shape[2] == P_max
    dev = partial_target.device
    if idx is None:
        idx = torch.empty((n_rows, k), dtype=torch.int32, device=dev)
    if n_sel is None:
        n_sel = torch.empty((n_rows,), dtype=torch.int32, device=dev)
    if workspace is None:
        nb = ctypes.c_size_t(0)
        _check(lib.vsd_select_hybrid_workspace_size(n_rows, P_max, ctypes.byref(nb)),
               "vsd_select_hybrid_workspace_size")
        workspace = _workspace(int(nb.value), dev, "select_hybrid")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.vsd_select_topk_hybrid(n_rows, Hkv_t, _ptr(partial_target), Hkv_d,
                                    _ptr(partial_draft), _ptr(prefix_len), P_max, int(k), int(m),
                                    int(n_sink), int(n_recent), _ptr(idx), _ptr(n_sel),
                                    _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "vsd_select_topk_hybrid")
    return idx, n_sel


def page_blocks(P_max: int) -> int:
    """Pages of 16 tokens covering a prefix of P_max tokens."""
    return (int(P_max) + 15) // 16


def vsd_page_key_means(k_cache, block_table, prefix_len, *, B: int, page_blocks_max: int,
                       page_begin=None, page_means=None, stream=None):
    """Mean key of every prefix page: fp32 [B, Hkv, page_blocks_max, d] (pages from
    page_begin[b], default 0, to ceil(P_b / 16) are written).  Returns page_means."""
    lib = load()
    _need(prefix_len, torch.int32, "prefix_len")
    if page_begin is not None:
        _need(page_begin, torch.int32, "page_begin")
    Hkv, d = int(k_cache.shape[1]), int(k_cache.shape[3])
    geom = geom_for(B, Hkv, k_cache, block_table)
    if page_means is None:
        page_means = torch.zeros((B, Hkv, page_blocks_max, d), dtype=torch.float32,
                                 device=k_cache.device)
    rc = lib.vsd_page_key_means(ctypes.byref(geom), _ptr(k_cache), _ptr(block_table),
                                _ptr(prefix_len), _ptr(page_begin), int(page_blocks_max),
                                _ptr(page_means), _stream(stream))
    _check(rc, "vsd_page_key_means")
    return page_means


def vsd_block_topk(q, page_means, prefix_len, *, kb: int, scale: float, k_cache=None,
                   block_table=None, scores=None, blocks=None, stream=None):
    """Per-query page scores fp32 [B, R, Hq, page_blocks_max] and the kb best pages of
    every (b, t, h), ascending and padded with -1: int32 [B, R, Hq, kb].  q: bf16
    [B, R, Hq, d]; page_means from vsd_page_key_means.  Returns (scores, blocks)."""
    lib = load()
    B, R, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    _need(page_means, torch.float32, "page_means")
    _need(prefix_len, torch.int32, "prefix_len")
    Hkv, nblk = int(page_means.shape[1]), int(page_means.shape[2])
    geom = Geom(B, Hq, Hkv, d, 16, 1, 1)
    if k_cache is not None:
        geom = geom_for(B, Hq, k_cache, block_table)
    dev = q.device
    if scores is None:
        scores = torch.zeros((B, R, Hq, nblk), dtype=torch.float32, device=dev)
    if blocks is None:
        blocks = torch.empty((B, R, Hq, kb), dtype=torch.int32, device=dev)
    rc = lib.vsd_block_topk(ctypes.byref(geom), R, _ptr(q), _ptr(page_means), _ptr(prefix_len),
                            nblk, int(kb), float(scale), _ptr(scores), _ptr(blocks),
                            _stream(stream))
    _check(rc, "vsd_block_topk")
    return scores, blocks


HIST_BINS = 4096


def vsd_verify_attn_collect_scored(q, k_cache, v_cache, block_table, prefix_len, *, P_max: int,
                                   scale: float, row0: int = 0, row1: Optional[int] = None,
                                   logits=None, partial=None, score=None, score_hist=None,
                                   n_sink: int = 0, n_recent: int = 0, flags: int = 0,
                                   k_new=None, v_new=None, out=None, workspace=None, stream=None):
    """Verification with Collect-2-Query that also sums the partial scores over the KV
    groups (score fp32 [B, P_max]) and counts the level-0 histogram (uint32-valued int32
    [B, 4096]) of the selection's candidates (the n_sink first and n_recent last prefix
    positions left out).  flags: 0 or VERIFY_EARLY_PREFETCH.  k_new, v_new: bf16
    [B, R, Hkv, d] or None: the verify block's keys and values, stored into the caches at
    P_b .. P_b + R - 1 by the call itself.  Returns (out, logits, partial, score,
    score_hist)."""
    lib = load()
    B, R, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    for name, x in (("k_new", k_new), ("v_new", v_new)):
        if x is not None:
            _need(x, torch.bfloat16, name)
    geom = geom_for(B, Hq, k_cache, block_table)
    if row1 is None:
        row1 = R - 1
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if partial is None:
        partial = torch.empty((B, geom.Hkv, P_max), dtype=torch.float32, device=dev)
    if score is None:
        score = torch.empty((B, P_max), dtype=torch.float32, device=dev)
    if score_hist is None:
        score_hist = torch.empty((B, HIST_BINS), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _workspace(vsd_verify_workspace_size(geom, R, P_max), dev, "verify")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.vsd_verify_attn_collect_scored(ctypes.byref(geom), R, _ptr(q), _ptr(k_cache),
                                            _ptr(v_cache), _ptr(block_table), _ptr(prefix_len),
                                            int(row0), int(row1), int(P_max), float(scale),
                                            _ptr(logits), _ptr(partial), _ptr(score),
                                            _ptr(score_hist), int(n_sink), int(n_recent),
                                            int(flags), _ptr(k_new), _ptr(v_new), _ptr(out),
                                            _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "vsd_verify_attn_collect_scored")
    return out, logits, partial, score, score_hist


def vsd_select_topk_scored(score, score_hist, prefix_len, *, k: int, n_sink: int, n_recent: int,
                           idx=None, n_sel=None, stream=None):
    """The protected top-k from an aggregated score [n_rows, P_max] and its histogram
    (from vsd_verify_attn_collect_scored).  Returns (idx [n_rows, k], n_sel)."""
    lib = load()
    _need(score, torch.float32, "score")
    n_rows, P_max = score.shape
    dev = score.device
    if idx is None:
        idx = torch.empty((n_rows, k), dtype=torch.int32, device=dev)
    if n_sel is None:
        n_sel = torch.empty((n_rows,), dtype=torch.int32, device=dev)
    rc = lib.vsd_select_topk_scored(int(n_rows), _ptr(score), _ptr(score_hist), _ptr(prefix_len),
                                    int(P_max), int(k), int(n_sink), int(n_recent), _ptr(idx),
                                    _ptr(n_sel), _stream(stream))
    _check(rc, "vsd_select_topk_scored")
    return idx, n_sel


def vsd_copy(dst, src, stream=None):
    """dst <- src (same byte size, a multiple of 16) by a kernel; either tensor may be in
    pinned host memory."""
    lib = load()
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("vsd_copy: size mismatch")
    _check(lib.vsd_copy(_ptr(dst), _ptr(src), nbytes, _stream(stream)), "vsd_copy")
    return dst


def vsd_append_kv(k_new, v_new, k_cache, v_cache, block_table, pos_base, *, pos_offset: int = 0,
                  stream=None):
    """Store K/V rows k_new, v_new: bf16 [B, n_new, Hkv, d] at positions
    pos_base[b] + pos_offset + t of each sequence (through the block table)."""
    lib = load()
    _need(k_new, torch.bfloat16, "k_new")
    _need(v_new, torch.bfloat16, "v_new")
    _need(pos_base, torch.int32, "pos_base")
    B, n_new = int(k_new.shape[0]), int(k_new.shape[1])
    if tuple(v_new.shape) != tuple(k_new.shape):
        raise ValueError("k_new and v_new shapes differ")
    geom = geom_for(B, int(k_cache.shape[1]), k_cache, block_table)
    rc = lib.vsd_append_kv(ctypes.byref(geom), n_new, _ptr(k_new), _ptr(v_new), _ptr(block_table),
                           _ptr(pos_base), int(pos_offset), _ptr(k_cache), _ptr(v_cache),
                           _stream(stream))
    _check(rc, "vsd_append_kv")


def vsd_advance_lengths(accepted, prefix_len, tail_start, seq_len, *, max_prefix: int,
                        prefix_copies=None, stream=None):
    """After a verification that accepted accepted[b] drafts: prefix_len += accepted + 1,
    tail_start = the old prefix, seq_len[i] = old prefix + accepted + 2 + i, and every row
    of prefix_copies ([n_copies, B]) = the new prefix.  All int32 device tensors."""
    lib = load()
    for t, name in ((accepted, "accepted"), (prefix_len, "prefix_len"),
                    (tail_start, "tail_start"), (seq_len, "seq_len")):
        _need(t, torch.int32, name)
    B = int(prefix_len.shape[0])
    gamma = int(seq_len.shape[0])
    n_copies = 0
    if prefix_copies is not None:
        _need(prefix_copies, torch.int32, "prefix_copies")
        n_copies = prefix_copies.numel() // max(B, 1)
    rc = lib.vsd_advance_lengths(B, gamma, _ptr(accepted), int(max_prefix), _ptr(prefix_len),
                                 _ptr(tail_start), _ptr(seq_len), n_copies, _ptr(prefix_copies),
                                 _stream(stream))
    _check(rc, "vsd_advance_lengths")


def vsd_sparse_decode_attn_step(q, k_cache, v_cache, block_table, idx, n_sel, tail_start, seq_len,
                                *, scale: float, max_tail: int, k_new=None, v_new=None,
                                sel_rows=None, flags: int = 0, out=None, workspace=None,
                                stream=None):
    """A draft step of a decode loop: the step's input token (k_new, v_new: bf16
    [B, Hkv, d]) is stored at seq_len - 1 and attended; sel_rows (int32 [B, k_max]) caches
    the selection's cache rows (STEP_RECORD_ROWS writes them, STEP_REUSE_ROWS reads
    them); STEP_EARLY_GATHER gathers before waiting for the preceding kernel (see
    include/vsd.h for what the caller promises with it)."""
    lib = load()
    B, Hq, d = q.shape
    _need(q, torch.bfloat16, "q")
    _need(tail_start, torch.int32, "tail_start")
    _need(seq_len, torch.int32, "seq_len")
    if k_new is not None:
        _need(k_new, torch.bfloat16, "k_new")
        _need(v_new, torch.bfloat16, "v_new")
    if sel_rows is not None:
        _need(sel_rows, torch.int32, "sel_rows")
    geom = geom_for(B, Hq, k_cache, block_table)
    k_max = 0 if idx is None else int(idx.shape[1])
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = _workspace(vsd_sparse_workspace_size(geom, k_max, max_tail), q.device,
                               "sparse:%d" % (geom.B * geom.Hkv))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.vsd_sparse_decode_attn_step(ctypes.byref(geom), _ptr(q), _ptr(k_new), _ptr(v_new),
                                         _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                         _ptr(idx), _ptr(n_sel), k_max, _ptr(tail_start),
                                         _ptr(seq_len), int(max_tail), _ptr(sel_rows),
                                         int(flags), float(scale), _ptr(out), _ptr(workspace),
                                         ws_bytes, _stream(stream))
    _check(rc, "vsd_sparse_decode_attn_step")
    return out


# ------------------------------------------------------------------ 8-bit cache
# These calls are made once per layer and step, so their checks are one comparison per
# property and tensor on the way through; _refuse says afterwards what was wrong.
_F8, _BF16, _F32, _I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32


def _refuse(*wanted) -> None:
    """Raise what is wrong with the first of (tensor, dtype, shape, device, name) that is
    not as wanted."""
    for t, dtype, shape, dev, name in wanted:
        if t is None:
            continue
        _need(t, dtype, name)
        if tuple(t.shape) != tuple(shape):
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        if t.get_device() != dev:
            raise ValueError("%s is on another device" % name)
    raise ValueError("tensors do not fit together")


def _cuda_index(t, dtype, name: str) -> int:
    """The device of a call's first tensor."""
    dev = t.get_device()
    if dev < 0:
        _need(t, dtype, name)
    return dev


def _is(t, dtype, numel: int, dim: int, dev: int) -> bool:
    return t.dtype is dtype and t.numel() == numel and t.dim() == dim and \
        t.get_device() == dev and t.is_contiguous()


def _cache_shape(k_cache, v_cache, k_scale, v_scale, dev):
    """The shape (num_blocks, Hkv, 16, d) of an 8-bit cache: float8_e4m3fn codes and
    float32 scales [num_blocks, Hkv] on device `dev`."""
    shape = k_cache.shape
    if len(shape) == 4:
        n = shape[0] * shape[1]
        if k_cache.dtype is _F8 and v_cache.dtype is _F8 and v_cache.shape == shape and \
                k_cache.is_contiguous() and v_cache.is_contiguous() and \
                k_cache.get_device() == dev and v_cache.get_device() == dev and \
                k_scale.shape == v_scale.shape == shape[:2] and \
                _is(k_scale, _F32, n, 2, dev) and _is(v_scale, _F32, n, 2, dev):
            return shape
    _refuse((k_cache, _F8, shape if len(shape) == 4 else ("num_blocks", "Hkv", 16, "d"), dev, "k_cache"),
            (v_cache, _F8, shape, dev, "v_cache"), (k_scale, _F32, shape[:2], dev, "k_scale"),
            (v_scale, _F32, shape[:2], dev, "v_scale"))


def _elsewhere(dev: int) -> bool:
    """Whether a call's tensors are on another device than the current one (the library
    launches on the current device)."""
    return dev >= 0 and dev != torch._C._cuda_getDevice()


def _empty(stream, shape, dtype, dev, make=torch.empty):
    """What a call allocates (outputs, its scratch) comes from torch's allocator tied to
    the stream that the call runs on: calls on other streams, and captured graphs, get
    memory of their own, and it goes back in stream order."""
    if stream is None:
        return make(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=dev)


def _raw_stream(stream, dev: int) -> int:
    """The cudaStream_t of a call (torch's own accessor: a Stream object costs 3 us)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


@functools.lru_cache(maxsize=512)
def _quant_plan(call: str, dev: int, x: int, y: int, B: int, Hq: int, Hkv: int, d: int, page: int,
                max_blocks: int, num_blocks: int):
    """(geometry, its address, workspace bytes) of a call, kept for the next one of the same
    shape.  `call` names the size query, "" for calls without a workspace."""
    geom = Geom(B, Hq, Hkv, d, page, max_blocks, num_blocks)
    nbytes = ctypes.c_size_t(0)
    if call:
        _check(getattr(load(), call)(ctypes.addressof(geom), x, y, ctypes.byref(nbytes)), call)
    return geom, ctypes.addressof(geom), int(nbytes.value)


# Scratch of the current streams' eager calls, by (device, stream): (tensor, address, bytes).
# The calls of one stream run one after the other and ignore what it holds, so one buffer
# serves them all (an allocation between two launches takes 6 us).
_stream_scratch = {}
_PER_THREAD_STREAM = 2  # cudaStreamPerThread: one handle for a stream of every host thread


def _workspace_of(workspace, nbytes: int, stream, dev: int):
    """(the tensor that keeps it alive, address, bytes) of a call's scratch.  A captured call,
    and one that names its stream, gets memory of its own."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(dev)
            if raw != _PER_THREAD_STREAM and not torch._C._cuda_isCurrentStreamCapturing():
                kept = _stream_scratch.get((dev, raw))
                if kept is None or kept[2] < nbytes:
                    # (the smaller one goes back to the allocator in stream order)
                    new = torch.empty(nbytes, dtype=torch.uint8, device=dev)
                    kept = _stream_scratch[(dev, raw)] = (new, new.data_ptr(), nbytes)
                return kept
        workspace = _empty(stream, nbytes, torch.uint8, dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the call's device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _rows_plan(k_rows, v_rows, names, k_cache, v_cache, k_scale, v_scale, block_table, pos_base,
               n_valid, dev):
    """The checks that storing and reading rows share, and the geometry."""
    NB, Hkv, page, d = _cache_shape(k_cache, v_cache, k_scale, v_scale, dev)
    rows = k_rows.shape
    B, width = rows[0], block_table.shape[-1]
    if not (len(rows) == 4 and rows[2] == Hkv and rows[3] == d and
            _is(k_rows, _BF16, k_rows.numel(), 4, dev) and _is(v_rows, _BF16, k_rows.numel(), 4, dev) and
            v_rows.shape == rows and _is(block_table, _I32, B * width, 2, dev) and
            _is(pos_base, _I32, B, 1, dev) and (n_valid is None or _is(n_valid, _I32, B, 1, dev))):
        want = (B, rows[1] if len(rows) == 4 else "n", Hkv, d)
        _refuse((k_rows, _BF16, want, dev, names[0]), (v_rows, _BF16, want, dev, names[1]),
                (block_table, _I32, (B, width), dev, "block_table"), (pos_base, _I32, (B,), dev, "pos_base"),
                (n_valid, _I32, (B,), dev, "n_valid"))
    return _quant_plan("", dev, 0, 0, B, Hkv, Hkv, d, page, width, NB)


def vsd_append_kv_quant(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table, pos_base, *,
                        pos_offset: int = 0, n_valid=None, stream=None) -> None:
    """Quantise and store K/V rows k_new, v_new (bf16 [B, n_new, Hkv, d]) at positions
    pos_base[b] + pos_offset + t, t < n_valid[b] (None: all), of an 8-bit cache
    (float8_e4m3fn [num_blocks, Hkv, 16, d], scales float32 [num_blocks, Hkv]).  Rows are
    appended in order: a page whose slot 0 is written starts afresh, otherwise its earlier
    rows are kept (requantised when its scale has to grow)."""
    dev = _cuda_index(k_new, _BF16, "k_new")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return vsd_append_kv_quant(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table,
                                       pos_base, pos_offset=pos_offset, n_valid=n_valid, stream=stream)
    geom = _rows_plan(k_new, v_new, ("k_new", "v_new"), k_cache, v_cache, k_scale, v_scale, block_table,
                      pos_base, n_valid, dev)
    _check((_lib or load()).vsd_append_kv_quant(
        geom[1], k_new.shape[1], k_new.data_ptr(), v_new.data_ptr(), block_table.data_ptr(),
        pos_base.data_ptr(), pos_offset, None if n_valid is None else n_valid.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        _raw_stream(stream, dev)), "vsd_append_kv_quant")


def vsd_read_kv_quant(k_cache, v_cache, k_scale, v_scale, block_table, pos_base, *, n: int,
                      pos_offset: int = 0, n_valid=None, k_out=None, v_out=None, stream=None):
    """The rows at positions pos_base[b] + pos_offset + t, t < n_valid[b] (None: n), of an
    8-bit cache as bf16 [B, n, Hkv, d].  Rows behind n_valid are left as they were in
    k_out, v_out (zeros when allocated here).  Returns (k_out, v_out)."""
    dev = _cuda_index(k_cache, _F8, "k_cache")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return vsd_read_kv_quant(k_cache, v_cache, k_scale, v_scale, block_table, pos_base, n=n,
                                     pos_offset=pos_offset, n_valid=n_valid, k_out=k_out, v_out=v_out,
                                     stream=stream)
    if k_out is None or v_out is None:
        shape = (pos_base.shape[0], n, k_cache.shape[1], k_cache.shape[-1])
        make = torch.empty if n_valid is None else torch.zeros
        k_out = _empty(stream, shape, _BF16, dev, make) if k_out is None else k_out
        v_out = _empty(stream, shape, _BF16, dev, make) if v_out is None else v_out
    geom = _rows_plan(k_out, v_out, ("k_out", "v_out"), k_cache, v_cache, k_scale, v_scale, block_table,
                      pos_base, n_valid, dev)
    if k_out.shape[1] != n:
        raise ValueError("k_out and v_out must be [B, n, Hkv, d]")
    _check((_lib or load()).vsd_read_kv_quant(
        geom[1], n, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        block_table.data_ptr(), pos_base.data_ptr(), pos_offset,
        None if n_valid is None else n_valid.data_ptr(), k_out.data_ptr(), v_out.data_ptr(),
        _raw_stream(stream, dev)), "vsd_read_kv_quant")
    return k_out, v_out


def vsd_verify_quant_workspace_size(geom: Geom, R: int, P_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().vsd_verify_quant_workspace_size(ctypes.addressof(geom), int(R), int(P_max),
                                                  ctypes.byref(out)),
           "vsd_verify_quant_workspace_size")
    return int(out.value)


def _address(t):
    return None if t is None else t.data_ptr()


def _verify_quant(q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, P_max, scale,
                  row0, row1, logits, partial, score, score_hist, n_sink, n_recent, out,
                  workspace, stream, collect, scored):
    dev = _cuda_index(q, _BF16, "q")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return _verify_quant(q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, P_max,
                                 scale, row0, row1, logits, partial, score, score_hist, n_sink,
                                 n_recent, out, workspace, stream, collect, scored)
    NB, Hkv, page, d = _cache_shape(k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 4:
        raise ValueError("q must be [B, R, Hq, d]")
    B, R, Hq, dq = q.shape
    width = block_table.shape[-1]
    if out is None:
        out = _empty(stream, q.shape, _BF16, dev)
    if collect and logits is None:
        logits = _empty(stream, (B, 2, Hq, P_max), _F32, dev)
    if (collect or scored) and partial is None:
        partial = _empty(stream, (B, Hkv, P_max), _F32, dev)
    if scored and score is None:
        score = _empty(stream, (B, P_max), _F32, dev)
    if scored and score_hist is None:
        score_hist = _empty(stream, (B, HIST_BINS), _I32, dev)
    if not (dq == d and _is(q, _BF16, q.numel(), 4, dev) and _is(out, _BF16, q.numel(), 4, dev) and
            out.shape == q.shape and _is(block_table, _I32, B * width, 2, dev) and
            _is(prefix_len, _I32, B, 1, dev) and
            (logits is None or logits.shape == (B, 2, Hq, P_max) and _is(logits, _F32, logits.numel(), 4, dev)) and
            (partial is None or partial.shape == (B, Hkv, P_max) and _is(partial, _F32, partial.numel(), 3, dev)) and
            (score is None or score.shape == (B, P_max) and _is(score, _F32, score.numel(), 2, dev)) and
            (score_hist is None or score_hist.shape == (B, HIST_BINS) and _is(score_hist, _I32, B * HIST_BINS, 2, dev))):
        _refuse((q, _BF16, (B, R, Hq, d), dev, "q"), (out, _BF16, (B, R, Hq, d), dev, "out"),
                (block_table, _I32, (B, width), dev, "block_table"),
                (prefix_len, _I32, (B,), dev, "prefix_len"), (logits, _F32, (B, 2, Hq, P_max), dev, "logits"),
                (partial, _F32, (B, Hkv, P_max), dev, "partial"), (score, _F32, (B, P_max), dev, "score"),
                (score_hist, _I32, (B, HIST_BINS), dev, "score_hist"))
    plan = _quant_plan("vsd_verify_quant_workspace_size", dev, R, P_max, B, Hq, Hkv, d, page, width, NB)
    keep, wp, wb = _workspace_of(workspace, plan[2], stream, dev)
    _check((_lib or load()).vsd_verify_attn_collect_quant(
        plan[1], R, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), block_table.data_ptr(), prefix_len.data_ptr(), row0,
        R - 1 if row1 is None else row1, P_max, scale, _address(logits), _address(partial),
        _address(score), _address(score_hist), n_sink, n_recent, out.data_ptr(), wp, wb,
        _raw_stream(stream, dev)), "vsd_verify_attn_collect_quant")
    return out, logits, partial, score, score_hist


def vsd_verify_attn_collect_quant(q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len,
                                  *, P_max: int, scale: float, row0: int = 0,
                                  row1: Optional[int] = None, logits=None, partial=None, out=None,
                                  collect: bool = True, workspace=None, stream=None):
    """Verification attention + Collect-2-Query over an 8-bit cache (float8_e4m3fn
    [num_blocks, Hkv, 16, d] with scales float32 [num_blocks, Hkv]); with R = 1 the
    attention of single tokens.  Returns (out, logits, partial)."""
    return _verify_quant(q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, P_max,
                         scale, row0, row1, logits, partial, None, None, 0, 0, out, workspace,
                         stream, collect, False)[:3]


def vsd_verify_attn_collect_scored_quant(q, k_cache, v_cache, k_scale, v_scale, block_table,
                                         prefix_len, *, P_max: int, scale: float, row0: int = 0,
                                         row1: Optional[int] = None, logits=None, partial=None,
                                         score=None, score_hist=None, n_sink: int = 0,
                                         n_recent: int = 0, out=None, workspace=None, stream=None):
    """vsd_verify_attn_collect_quant that also writes the aggregated score and its
    histogram for vsd_select_topk_scored (logits are written when given).  Returns (out,
    logits, partial, score, score_hist)."""
    return _verify_quant(q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, P_max,
                         scale, row0, row1, logits, partial, score, score_hist, n_sink, n_recent,
                         out, workspace, stream, False, True)


def vsd_sparse_quant_workspace_size(geom: Geom, k_max: int, max_tail: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().vsd_sparse_quant_workspace_size(ctypes.addressof(geom), int(k_max),
                                                  int(max_tail), ctypes.byref(out)),
           "vsd_sparse_quant_workspace_size")
    return int(out.value)


def vsd_sparse_decode_attn_quant(q, k_cache, v_cache, k_scale, v_scale, block_table, idx, n_sel,
                                 tail_start, seq_len, *, scale: float, max_tail: int, out=None,
                                 workspace=None, stream=None):
    """Sparse draft-step attention over an 8-bit cache.  q: bf16 [B, Hq, d]; idx: int32
    [B, k_max] and n_sel: int32 [B], or both None.  Returns out."""
    dev = _cuda_index(q, _BF16, "q")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return vsd_sparse_decode_attn_quant(q, k_cache, v_cache, k_scale, v_scale, block_table, idx,
                                                n_sel, tail_start, seq_len, scale=scale,
                                                max_tail=max_tail, out=out, workspace=workspace,
                                                stream=stream)
    NB, Hkv, page, d = _cache_shape(k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, d]")
    B, Hq, dq = q.shape
    width = block_table.shape[-1]
    if (idx is None) != (n_sel is None):
        raise ValueError("idx and n_sel go together")
    k_max = 0 if idx is None else idx.shape[-1]
    if out is None:
        out = _empty(stream, q.shape, _BF16, dev)
    if not (dq == d and _is(q, _BF16, q.numel(), 3, dev) and _is(out, _BF16, q.numel(), 3, dev) and
            out.shape == q.shape and _is(block_table, _I32, B * width, 2, dev) and
            _is(tail_start, _I32, B, 1, dev) and _is(seq_len, _I32, B, 1, dev) and
            (idx is None or _is(idx, _I32, B * k_max, 2, dev) and _is(n_sel, _I32, B, 1, dev))):
        _refuse((q, _BF16, (B, Hq, d), dev, "q"), (out, _BF16, (B, Hq, d), dev, "out"),
                (block_table, _I32, (B, width), dev, "block_table"),
                (tail_start, _I32, (B,), dev, "tail_start"), (seq_len, _I32, (B,), dev, "seq_len"),
                (idx, _I32, (B, k_max), dev, "idx"), (n_sel, _I32, (B,), dev, "n_sel"))
    plan = _quant_plan("vsd_sparse_quant_workspace_size", dev, k_max, max_tail, B, Hq, Hkv, d, page,
                       width, NB)
    keep, wp, wb = _workspace_of(workspace, plan[2], stream, dev)
    _check((_lib or load()).vsd_sparse_decode_attn_quant(
        plan[1], q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), block_table.data_ptr(), _address(idx), _address(n_sel), k_max,
        tail_start.data_ptr(), seq_len.data_ptr(), max_tail, scale, out.data_ptr(), wp, wb,
        _raw_stream(stream, dev)), "vsd_sparse_decode_attn_quant")
    return out
