"""Python binding of ``libbsa.so``: block-sparse causal attention on B200
(forward, gradients, selected-page decode, attention of drafted token trees and
cache eviction by attention weight).

Argument marshalling only.  Every step of the computation runs in the
library's CUDA kernel or its host layout compiler; this module converts Python
values and torch tensors to the C ABI declared in ``include/bsa.h`` and turns
non-zero status codes into :class:`BsaError`.  There is no fallback: if the
shared library is missing or cannot be loaded, every call raises.

Names follow the C ABI: ``bsa_build_layout``, ``bsa_layout_csr``,
``bsa_layout_csc``, ``bsa_layout_order``, ``bsa_layout_segments``,
``bsa_forward``, ``bsa_forward_noalloc``, ``bsa_backward``, ``bsa_decode``,
``bsa_attention_weights``, ``bsa_decode_weights``, ``bsa_evict``,
``bsa_decode_tree``, ``bsa_get_status``, ``bsa_debug_timeout_probe``,
``bsa_free`` and ``bsa_last_error``; the ``Layout`` class, ``attention``,
``attention_backward``, ``decode``, ``attention_weights``, ``decode_weights``,
``evict`` and ``decode_tree`` are conveniences over them.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading

import numpy as np

from .workloads import (PATTERN_BAND_GLOBAL, PATTERN_DYADIC, PATTERN_RANDOM,  # noqa: F401
                        PATTERN_EXPLICIT)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsa.so")

BSA_OK = 0
STATUS_NAMES = {0: "BSA_OK", 1: "BSA_ERR_INVALID_ARG", 2: "BSA_ERR_SHAPE", 3: "BSA_ERR_UNSUPPORTED",
                4: "BSA_ERR_NONCAUSAL", 5: "BSA_ERR_CUDA", 6: "BSA_ERR_OOM",
                7: "BSA_ERR_DEVICE_TIMEOUT"}

EXPORTED = ["bsa_build_layout", "bsa_layout_csr", "bsa_layout_csc", "bsa_layout_order", "bsa_layout_work",
            "bsa_layout_segments", "bsa_forward", "bsa_forward_host", "bsa_forward_noalloc", "bsa_backward",
            "bsa_decode", "bsa_attention_weights_workspace_bytes", "bsa_attention_weights",
            "bsa_decode_weights_workspace_bytes", "bsa_decode_weights", "bsa_evict_workspace_bytes", "bsa_evict",
            "bsa_decode_tree_workspace_bytes", "bsa_decode_tree",
            "bsa_bsbr_workspace_bytes", "bsa_bsbr_retrieval", "bsa_get_status", "bsa_debug_timeout_probe",
            "bsa_free", "bsa_last_error"]


class BsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")


class bsa_pattern(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("window", ctypes.c_int32),
                ("global_first", ctypes.c_int32), ("dyadic_kmin", ctypes.c_int32),
                ("density", ctypes.c_double), ("seed", ctypes.c_uint64),
                ("mask", ctypes.POINTER(ctypes.c_uint8))]


_lib = None
_lib_lock = threading.Lock()


def load_library(path: str = LIB_PATH):
    """Load (once) and return the ctypes handle; raises if the library is absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libbsa.so not found at {path}; build it with "
                               "`python -m block_sparse_long_bsa_b200.build`")
        lib = ctypes.CDLL(path)
        P, I, U64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_float
        lib.bsa_build_layout.argtypes = [ctypes.POINTER(bsa_pattern), I, I, I, I, ctypes.POINTER(P)]
        lib.bsa_build_layout.restype = I
        lib.bsa_layout_csr.argtypes = [P, ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                       ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                       ctypes.POINTER(I), ctypes.POINTER(I)]
        lib.bsa_layout_csr.restype = I
        lib.bsa_layout_csc.argtypes = [P, ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                       ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                       ctypes.POINTER(I), ctypes.POINTER(I)]
        lib.bsa_layout_csc.restype = I
        lib.bsa_layout_order.argtypes = [P, ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                         ctypes.POINTER(I)]
        lib.bsa_layout_order.restype = I
        lib.bsa_layout_work.argtypes = [P, ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                        ctypes.POINTER(I)]
        lib.bsa_layout_work.restype = I
        lib.bsa_forward.argtypes = [P, P, P, P, I, I, I, I, I, F, P, P, P]
        lib.bsa_forward.restype = I
        lib.bsa_forward_noalloc.argtypes = [P, P, P, P, I, I, I, I, I, F, P, P, P]
        lib.bsa_forward_noalloc.restype = I
        lib.bsa_forward_host.argtypes = [P, P, P, P, I, I, I, I, I, F, P, P, P, P, P, P, P, I, P]
        lib.bsa_forward_host.restype = I
        lib.bsa_decode.argtypes = [P, P, P, P, I, I, P, P, I, I, I, I, F, P, P, P]
        lib.bsa_decode.restype = I
        S = ctypes.c_size_t
        lib.bsa_attention_weights_workspace_bytes.argtypes = [P, I, I]
        lib.bsa_attention_weights_workspace_bytes.restype = S
        lib.bsa_attention_weights.argtypes = [P, P, P, P, I, I, I, I, I, F, P, S, P, S, P]
        lib.bsa_attention_weights.restype = I
        lib.bsa_decode_weights_workspace_bytes.argtypes = [P, I, I, I, I]
        lib.bsa_decode_weights_workspace_bytes.restype = S
        lib.bsa_decode_weights.argtypes = [P, P, P, P, I, I, P, P, I, I, I, I, F, P, P, P, S, P, S, P]
        lib.bsa_decode_weights.restype = I
        lib.bsa_evict_workspace_bytes.argtypes = [P, I, I, I]
        lib.bsa_evict_workspace_bytes.restype = S
        lib.bsa_evict.argtypes = [P, P, P, I, I, P, P, P, P, I, I, I, I, I, S, P, P, P, P, S, P]
        lib.bsa_evict.restype = I
        lib.bsa_decode_tree_workspace_bytes.argtypes = [P, I, I, I, I, I]
        lib.bsa_decode_tree_workspace_bytes.restype = S
        lib.bsa_decode_tree.argtypes = [P, P, P, P, P, P, I, I, P, P, P, I, I, I, I, I, F, P, P, P, S, P]
        lib.bsa_decode_tree.restype = I
        lib.bsa_backward.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, P, P, P]
        lib.bsa_backward.restype = I
        lib.bsa_layout_segments.argtypes = [P, ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                            ctypes.POINTER(ctypes.POINTER(ctypes.c_int32)),
                                            ctypes.POINTER(I), ctypes.POINTER(I)]
        lib.bsa_layout_segments.restype = I
        lib.bsa_bsbr_workspace_bytes.argtypes = [I, I, I, I]
        lib.bsa_bsbr_workspace_bytes.restype = ctypes.c_size_t
        lib.bsa_bsbr_retrieval.argtypes = [P, P, P, P, I, I, I, I, I, F, P, P, ctypes.c_size_t, P]
        lib.bsa_bsbr_retrieval.restype = I
        lib.bsa_get_status.argtypes = [P, P]
        lib.bsa_get_status.restype = I
        lib.bsa_debug_timeout_probe.argtypes = [P, I, U64, P]
        lib.bsa_debug_timeout_probe.restype = I
        lib.bsa_free.argtypes = [P]
        lib.bsa_free.restype = None
        lib.bsa_last_error.argtypes = []
        lib.bsa_last_error.restype = ctypes.c_char_p
        _lib = lib
        return lib


def bsa_last_error() -> str:
    msg = load_library().bsa_last_error()
    return msg.decode() if msg else ""


def _check(status: int):
    if status != BSA_OK:
        raise BsaError(status, bsa_last_error())


def _ptr(x) -> int:
    """Device/host address of a torch tensor, or an int passed through."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None            # torch's functions for the current stream's handle, once it runs CUDA


def _stream(s) -> int:
    global _raw_stream
    if s is None:
        if _raw_stream is not None:
            # the handle alone: building a Stream object takes several times as long
            return _raw_stream[0](_raw_stream[1]())
        try:
            import torch
            if torch.cuda.is_initialized():
                # torch's internal names; one that lacks them is asked for the Stream below
                current = getattr(torch._C, "_cuda_getCurrentRawStream", None)
                device = getattr(torch._C, "_cuda_getDevice", None)
                if current and device:
                    _raw_stream = current, device
                    return current(device())
            if torch.cuda.is_available():
                return torch.cuda.current_stream().cuda_stream
        except ImportError:
            pass
        return 0
    if isinstance(s, int):
        return s
    return s.cuda_stream


def bsa_build_layout(kind: int, n: int, B: int, layout_heads: int = 1, device: int = -1,
                     window: int = 0, global_first: int = 0, dyadic_kmin: int = 2,
                     density: float = 0.0, seed: int = 0, mask=None) -> int:
    """Compile a pattern; returns the opaque layout handle (an int)."""
    lib = load_library()
    spec = bsa_pattern(kind, window, global_first, dyadic_kmin, density, seed & ((1 << 64) - 1), None)
    keep = None
    if mask is not None:
        keep = np.ascontiguousarray(mask, dtype=np.uint8)
        spec.mask = keep.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8))
    out = ctypes.c_void_p()
    _check(lib.bsa_build_layout(ctypes.byref(spec), n, B, layout_heads, device, ctypes.byref(out)))
    return out.value


def bsa_layout_csc(layout: int):
    """Copies of the transposed layout (col_ptr, row_idx) as int32 numpy arrays."""
    lib = load_library()
    cp = ctypes.POINTER(ctypes.c_int32)()
    ri = ctypes.POINTER(ctypes.c_int32)()
    cols, nnz = ctypes.c_int(), ctypes.c_int()
    _check(lib.bsa_layout_csc(layout, ctypes.byref(cp), ctypes.byref(ri), ctypes.byref(cols),
                              ctypes.byref(nnz)))
    col_ptr = np.ctypeslib.as_array(cp, shape=(cols.value + 1,)).copy()
    row_idx = (np.ctypeslib.as_array(ri, shape=(nnz.value,)).copy() if nnz.value
               else np.zeros(0, np.int32))
    return col_ptr, row_idx


def bsa_layout_segments(layout: int):
    """Copies of the key/value-gradient work list: (seg_ptr [L+1], segs [count, 3])."""
    lib = load_library()
    sp = ctypes.POINTER(ctypes.c_int32)()
    sg = ctypes.POINTER(ctypes.c_int32)()
    lh, cnt = ctypes.c_int(), ctypes.c_int()
    _check(lib.bsa_layout_segments(layout, ctypes.byref(sp), ctypes.byref(sg), ctypes.byref(lh),
                                   ctypes.byref(cnt)))
    seg_ptr = np.ctypeslib.as_array(sp, shape=(lh.value + 1,)).copy()
    segs = (np.ctypeslib.as_array(sg, shape=(cnt.value * 3,)).copy().reshape(-1, 3) if cnt.value
            else np.zeros((0, 3), np.int32))
    return seg_ptr, segs


def bsa_layout_csr(layout: int):
    """Copies of (row_ptr, col_idx) as int32 numpy arrays."""
    lib = load_library()
    rp = ctypes.POINTER(ctypes.c_int32)()
    ci = ctypes.POINTER(ctypes.c_int32)()
    rows, nnz = ctypes.c_int(), ctypes.c_int()
    _check(lib.bsa_layout_csr(layout, ctypes.byref(rp), ctypes.byref(ci), ctypes.byref(rows),
                              ctypes.byref(nnz)))
    row_ptr = np.ctypeslib.as_array(rp, shape=(rows.value + 1,)).copy()
    col_idx = (np.ctypeslib.as_array(ci, shape=(nnz.value,)).copy() if nnz.value
               else np.zeros(0, np.int32))
    return row_ptr, col_idx


def bsa_layout_order(layout: int) -> np.ndarray:
    lib = load_library()
    od = ctypes.POINTER(ctypes.c_int32)()
    cnt = ctypes.c_int()
    _check(lib.bsa_layout_order(layout, ctypes.byref(od), ctypes.byref(cnt)))
    return np.ctypeslib.as_array(od, shape=(cnt.value,)).copy()


def bsa_layout_work(layout: int) -> np.ndarray:
    """The forward's work table as an int32 array [layout_heads * nb, 4]."""
    lib = load_library()
    wk = ctypes.POINTER(ctypes.c_int32)()
    cnt = ctypes.c_int()
    _check(lib.bsa_layout_work(layout, ctypes.byref(wk), ctypes.byref(cnt)))
    return np.ctypeslib.as_array(wk, shape=(cnt.value * 4,)).copy().reshape(cnt.value, 4)


def bsa_forward(q, k, v, layout: int, B: int, n: int, heads: int, kv_heads: int, d: int,
                scale: float, o, lse, stream=None) -> None:
    """Enqueue the forward on ``stream`` (default: torch's current stream)."""
    lib = load_library()
    _check(lib.bsa_forward(_ptr(q), _ptr(k), _ptr(v), layout, B, n, heads, kv_heads, d,
                           ctypes.c_float(scale), _ptr(o), _ptr(lse), _stream(stream)))


def bsa_forward_host(q_host, k_host, v_host, layout: int, B: int, n: int, heads: int, kv_heads: int, d: int,
                     scale: float, q, k, v, o, lse, o_host, lse_host, groups: int = 8, stream=None) -> None:
    """Forward from and to host memory (see include/bsa.h): copies in head
    groups overlap the other groups' compute; synchronise ``stream`` before
    reading ``o_host`` and ``lse_host``."""
    lib = load_library()
    _check(lib.bsa_forward_host(_ptr(q_host), _ptr(k_host), _ptr(v_host), layout, B, n, heads, kv_heads, d,
                                ctypes.c_float(scale), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                _ptr(o_host), _ptr(lse_host), groups, _stream(stream)))


def bsa_forward_noalloc(q, k, v, layout: int, B: int, n: int, heads: int, kv_heads: int, d: int,
                        scale: float, o, lse, stream=None) -> None:
    """Allocation-free forward (see include/bsa.h): ``layout`` may be host-only;
    its arrays are staged in the library's static device block."""
    lib = load_library()
    _check(lib.bsa_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), layout, B, n, heads, kv_heads, d,
                                   ctypes.c_float(scale), _ptr(o), _ptr(lse), _stream(stream)))


def bsa_decode(q, k_cache, v_cache, page_table, max_blocks: int, num_pages: int, positions,
               layout: int, batch: int, heads: int, kv_heads: int, d: int, scale: float,
               o, lse, stream=None) -> None:
    """Enqueue one selected-page decode step (see include/bsa.h)."""
    lib = load_library()
    _check(lib.bsa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), max_blocks,
                          num_pages, _ptr(positions), layout, batch, heads, kv_heads, d,
                          ctypes.c_float(scale), _ptr(o), _ptr(lse), _stream(stream)))


def bsa_backward(q, k, v, o, lse, dout, layout: int, B: int, n: int, heads: int, kv_heads: int,
                 d: int, scale: float, dq, dk, dv, workspace, stream=None) -> None:
    """Enqueue the gradients of the forward (see include/bsa.h)."""
    lib = load_library()
    _check(lib.bsa_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), layout, B, n,
                            heads, kv_heads, d, ctypes.c_float(scale), _ptr(dq), _ptr(dk), _ptr(dv),
                            _ptr(workspace), _stream(stream)))


def attention_backward(q, k, v, o, lse, dout, layout: "Layout", scale: float | None = None,
                       dq=None, dk=None, dv=None, workspace=None, stream=None):
    """torch convenience: the forward's tensors plus dout [heads, n, d] bf16;
    returns fp32 (dq, dk, dv), allocating what is not given."""
    import torch
    heads, n, d = q.shape
    kv_heads = k.shape[0]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    for t in (q, k, v, o, dout):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise BsaError(1, "q, k, v, o and dout must be contiguous bf16 tensors")
    if dq is None:
        dq = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty(k.shape, dtype=torch.float32, device=q.device)
    if dv is None:
        dv = torch.empty(v.shape, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty((heads, n), dtype=torch.float32, device=q.device)
    for t in (lse, dq, dk, dv, workspace):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise BsaError(1, "lse, dq, dk, dv and workspace must be contiguous float32 tensors")
    bsa_backward(q, k, v, o, lse, dout, layout.handle, layout.B, n, heads, kv_heads, d, scale,
                 dq, dk, dv, workspace, stream)
    return dq, dk, dv


def bsa_bsbr_workspace_bytes(n: int, B: int, kv_heads: int, d: int) -> int:
    return int(load_library().bsa_bsbr_workspace_bytes(n, B, kv_heads, d))


def bsa_bsbr_retrieval(q, k, v, layout: int, B: int, n: int, heads: int, kv_heads: int, d: int,
                       scale: float, o, workspace, workspace_bytes: int, stream=None) -> None:
    """Enqueue BSBR's between-chunk retrieval term, added to ``o`` (see include/bsa.h)."""
    lib = load_library()
    _check(lib.bsa_bsbr_retrieval(_ptr(q), _ptr(k), _ptr(v), layout, B, n, heads, kv_heads, d,
                                  ctypes.c_float(scale), _ptr(o), _ptr(workspace), workspace_bytes,
                                  _stream(stream)))


def bsbr_attention(q, k, v, layout: "Layout", scale: float | None = None, workspace=None, stream=None):
    """torch convenience: the whole BSBR attention output for a block-diagonal
    ``layout`` (within-chunk forward, then the retrieval term added in place)."""
    import torch
    heads, n, d = q.shape
    kv_heads = k.shape[0]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o, lse = attention(q, k, v, layout, scale=scale, stream=stream)
    need = bsa_bsbr_workspace_bytes(n, layout.B, kv_heads, d)
    if workspace is None:
        workspace = torch.empty((max(need, 16) + 15) // 16 * 4, dtype=torch.float32, device=q.device)
    bsa_bsbr_retrieval(q, k, v, layout.handle, layout.B, n, heads, kv_heads, d, scale, o, workspace,
                       workspace.numel() * workspace.element_size(), stream)
    return o, lse


def decode(q, k_cache, v_cache, page_table, positions, layout: "Layout", batch: int,
           scale: float | None = None, o=None, lse=None, stream=None):
    """torch convenience: q [batch*H, d]; caches [pages, H_kv, B, d] bf16;
    page_table [batch, max_blocks] and positions [batch] int32, all on the GPU."""
    import torch
    heads, d = q.shape
    kv_heads = k_cache.shape[1] * batch
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((heads,), dtype=torch.float32, device=q.device)
    for t in (q, k_cache, v_cache, o):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise BsaError(1, "q, caches and o must be contiguous bf16 tensors")
    for t in (page_table, positions):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise BsaError(1, "page_table and positions must be contiguous int32 tensors")
    bsa_decode(q, k_cache, v_cache, page_table, page_table.shape[1], k_cache.shape[0], positions,
               layout.handle, batch, heads, kv_heads, d, scale, o, lse, stream)
    return o, lse


def bsa_attention_weights_workspace_bytes(layout: int, heads: int, kv_heads: int) -> int:
    return int(load_library().bsa_attention_weights_workspace_bytes(layout, heads, kv_heads))


def bsa_attention_weights(q, k, lse, layout: int, B: int, n: int, heads: int, kv_heads: int, d: int,
                          scale: float, weights, weights_stride: int, workspace, workspace_bytes: int,
                          stream=None) -> None:
    """Enqueue the sum of the weights that a prompt's keys receive (see include/bsa.h)."""
    lib = load_library()
    _check(lib.bsa_attention_weights(_ptr(q), _ptr(k), _ptr(lse), layout, B, n, heads, kv_heads, d,
                                     scale, _ptr(weights), weights_stride, _ptr(workspace),
                                     workspace_bytes, _stream(stream)))


def bsa_decode_weights_workspace_bytes(layout: int, batch: int, heads: int, kv_heads: int, d: int) -> int:
    return int(load_library().bsa_decode_weights_workspace_bytes(layout, batch, heads, kv_heads, d))


def bsa_decode_weights(q, k_cache, v_cache, page_table, max_blocks: int, num_pages: int, positions, layout: int,
                       batch: int, heads: int, kv_heads: int, d: int, scale: float, o, lse, weights,
                       weights_stride: int, workspace, workspace_bytes: int, stream=None) -> None:
    """Enqueue one decode step that adds its weights up (see include/bsa.h)."""
    lib = load_library()
    _check(lib.bsa_decode_weights(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), max_blocks, num_pages,
                                  _ptr(positions), layout, batch, heads, kv_heads, d, scale, _ptr(o),
                                  _ptr(lse), _ptr(weights), weights_stride, _ptr(workspace), workspace_bytes,
                                  _stream(stream)))


def bsa_evict_workspace_bytes(layout: int, batch: int, kv_heads: int, budget: int) -> int:
    return int(load_library().bsa_evict_workspace_bytes(layout, batch, kv_heads, budget))


def bsa_evict(k_cache, v_cache, page_table, max_blocks: int, num_pages: int, lengths, weights, tokens, layout: int,
              batch: int, kv_heads: int, d: int, budget: int, recent: int, stride: int, weights_out, tokens_out,
              lengths_out, workspace, workspace_bytes: int, stream=None) -> None:
    """Enqueue the cut of a paged cache to a budget (see include/bsa.h)."""
    lib = load_library()
    _check(lib.bsa_evict(_ptr(k_cache), _ptr(v_cache), _ptr(page_table), max_blocks, num_pages, _ptr(lengths),
                         _ptr(weights), _ptr(tokens), layout, batch, kv_heads, d, budget, recent, stride,
                         _ptr(weights_out), _ptr(tokens_out), _ptr(lengths_out), _ptr(workspace), workspace_bytes,
                         _stream(stream)))


def bsa_decode_tree_workspace_bytes(layout: int, batch: int, heads: int, kv_heads: int, T: int, d: int) -> int:
    return int(load_library().bsa_decode_tree_workspace_bytes(layout, batch, heads, kv_heads, T, d))


def bsa_decode_tree(q, k_tree, v_tree, k_cache, v_cache, page_table, max_blocks: int, num_pages: int, lengths,
                    parents, layout: int, T: int, batch: int, heads: int, kv_heads: int, d: int, scale: float, o, lse,
                    workspace, workspace_bytes: int, stream=None) -> None:
    """Enqueue the attention of a tree of drafted tokens (see include/bsa.h)."""
    lib = load_library()
    _check(lib.bsa_decode_tree(_ptr(q), _ptr(k_tree), _ptr(v_tree), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                               max_blocks, num_pages, _ptr(lengths), _ptr(parents), layout, T, batch, heads, kv_heads,
                               d, scale, _ptr(o), _ptr(lse), _ptr(workspace), workspace_bytes,
                               _stream(stream)))


def _want(device: int, dtype, *checks) -> None:
    """Each (name, tensor, shape) contiguous, of the dtype and shape, on the
    device."""
    for name, t, shape in checks:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
            continue
        what = str(dtype).replace("torch.", "")
        if t.dtype is not dtype or not t.is_contiguous():
            raise BsaError(1, f"{name} must be a contiguous {what} tensor")
        if t.get_device() != device:
            raise BsaError(1, f"{name} is not on the layout's device (cuda:{device})")
        raise BsaError(2, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")


def _rows_of(layout: "Layout", rows: int, *checks) -> int:
    """The common distance between the rows of arrays [rows, >= n] whose last
    dimension is contiguous; ``checks`` of (name, tensor, dtype), None skipped."""
    n, stride = layout.n, None
    for name, t, dtype in checks:
        if t is None:
            continue
        shape = t.shape
        if t.dtype is not dtype or len(shape) != 2 or shape[0] != rows or shape[1] < n or t.stride(1) != 1:
            raise BsaError(2, f"{name} must be a {str(dtype).replace('torch.', '')} tensor of {rows} rows of at least "
                              f"{n}, contiguous along them")
        if t.get_device() != layout.device:
            raise BsaError(1, f"{name} is not on the layout's device (cuda:{layout.device})")
        here = t.stride(0) if rows > 1 else n
        if stride is not None and here != stride:
            raise BsaError(2, f"{name}: the arrays' rows must be equally far apart")
        stride = here
    if stride < n:
        raise BsaError(2, "rows overlap")
    return stride


def _on(stream):
    """Context in which torch allocates for ``stream`` (the current one if
    None), so that memory made here is not handed on while the work on the
    stream still uses it."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _workspace(layout: "Layout", workspace, stream, bytes_of, *sizes):
    """The given workspace, or a new one of ``bytes_of(handle, *sizes)`` bytes
    that torch holds for ``stream``; (tensor, bytes)."""
    if workspace is None:
        if layout.device < 0:
            raise BsaError(1, "layout was built host-only (device = -1)")
        import torch
        with _on(stream):
            workspace = torch.empty(max(bytes_of(layout.handle, *sizes), 16), dtype=torch.uint8,
                                    device=f"cuda:{layout.device}")
    elif not workspace.is_contiguous() or workspace.get_device() != layout.device:
        raise BsaError(1, f"workspace must be a contiguous tensor on cuda:{layout.device}")
    return workspace, workspace.nbytes


def attention_weights(q, k, lse, layout: "Layout", weights=None, scale: float | None = None, workspace=None,
                      stream=None):
    """torch convenience: adds to ``weights`` [kv_heads, >= n] fp32 (zeros when
    not given) what every key of the prompt q [heads, n, d], k [kv_heads, n, d]
    received under the forward's ``lse`` [heads, n]; returns it."""
    import torch
    heads, n, d = q.shape
    kv_heads = k.shape[0]
    dev, h = layout.device, layout.handle
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _want(dev, torch.bfloat16, ("q", q, (heads, layout.n, d)), ("k", k, (kv_heads, layout.n, d)))
    _want(dev, torch.float32, ("lse", lse, (heads, layout.n)))
    if weights is None:
        with _on(stream):
            weights = torch.zeros((kv_heads, n), dtype=torch.float32, device=q.device)
    stride = _rows_of(layout, kv_heads, ("weights", weights, torch.float32))
    workspace, size = _workspace(layout, workspace, stream, bsa_attention_weights_workspace_bytes, heads, kv_heads)
    _check(load_library().bsa_attention_weights(
        q.data_ptr(), k.data_ptr(), lse.data_ptr(), h, layout.B, n, heads, kv_heads, d, scale, weights.data_ptr(),
        stride, workspace.data_ptr(), size, _stream(stream)))
    return weights


def decode_weights(q, k_cache, v_cache, page_table, positions, layout: "Layout", batch: int, weights,
                   scale: float | None = None, o=None, lse=None, workspace=None, stream=None):
    """torch convenience: ``decode`` that also adds the step's weights to
    ``weights`` [batch * H_kv, >= n] fp32; returns (o, lse)."""
    import torch
    heads, d = q.shape
    pages, hkv = k_cache.shape[0], k_cache.shape[1]
    max_blocks = page_table.shape[-1]
    dev, h = layout.device, layout.handle
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None or lse is None:
        with _on(stream):
            o = torch.empty_like(q) if o is None else o
            lse = torch.empty((heads,), dtype=torch.float32, device=q.device) if lse is None else lse
    cache = (pages, hkv, layout.B, d)
    _want(dev, torch.bfloat16, ("q", q, (heads, d)), ("k_cache", k_cache, cache), ("v_cache", v_cache, cache),
          ("o", o, (heads, d)))
    _want(dev, torch.int32, ("page_table", page_table, (batch, max_blocks)), ("positions", positions, (batch,)))
    _want(dev, torch.float32, ("lse", lse, (heads,)))
    stride = _rows_of(layout, batch * hkv, ("weights", weights, torch.float32))
    workspace, size = _workspace(layout, workspace, stream, bsa_decode_weights_workspace_bytes, batch, heads,
                                 batch * hkv, d)
    _check(load_library().bsa_decode_weights(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), max_blocks, pages,
        positions.data_ptr(), h, batch, heads, batch * hkv, d, scale, o.data_ptr(), lse.data_ptr(), weights.data_ptr(),
        stride, workspace.data_ptr(), size, _stream(stream)))
    return o, lse


def evict(k_cache, v_cache, page_table, lengths, weights, layout: "Layout", budget: int, recent: int = 0,
          tokens=None, weights_out=None, tokens_out=None, lengths_out=None, workspace=None, stream=None):
    """torch convenience: cuts the caches [pages, H_kv, B, d] in place to
    ``budget`` tokens per key/value head by ``weights`` [batch * H_kv, >= n];
    returns (weights_out, tokens_out, lengths_out), allocating what is not
    given.  The outputs are not the inputs: they are the next call's inputs."""
    import torch
    batch = lengths.shape[0]
    pages, hkv, _, d = k_cache.shape
    rows, max_blocks = batch * hkv, page_table.shape[-1]
    dev, h = layout.device, layout.handle
    if weights_out is None or tokens_out is None or lengths_out is None:
        def like(dtype):
            # an output that is not given has its rows as far apart as the weights'
            return torch.empty_strided(weights.shape, weights.stride(), dtype=dtype, device=weights.device)

        with _on(stream):
            weights_out = like(torch.float32) if weights_out is None else weights_out
            tokens_out = like(torch.int32) if tokens_out is None else tokens_out
            lengths_out = torch.empty_like(lengths) if lengths_out is None else lengths_out
    cache = (pages, hkv, layout.B, d)
    _want(dev, torch.bfloat16, ("k_cache", k_cache, cache), ("v_cache", v_cache, cache))
    _want(dev, torch.int32, ("page_table", page_table, (batch, max_blocks)), ("lengths", lengths, (batch,)),
          ("lengths_out", lengths_out, (batch,)))
    stride = _rows_of(layout, rows, ("weights", weights, torch.float32), ("tokens", tokens, torch.int32),
                      ("weights_out", weights_out, torch.float32), ("tokens_out", tokens_out, torch.int32))
    workspace, size = _workspace(layout, workspace, stream, bsa_evict_workspace_bytes, batch, rows, budget)
    _check(load_library().bsa_evict(
        k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), max_blocks, pages, lengths.data_ptr(),
        weights.data_ptr(), 0 if tokens is None else tokens.data_ptr(), h, batch, rows, d, budget, recent, stride,
        weights_out.data_ptr(), tokens_out.data_ptr(), lengths_out.data_ptr(), workspace.data_ptr(), size,
        _stream(stream)))
    return weights_out, tokens_out, lengths_out


def decode_tree(q, k_tree, v_tree, k_cache, v_cache, page_table, lengths, parents, layout: "Layout",
                scale: float | None = None, o=None, lse=None, workspace=None, stream=None):
    """torch convenience: q [batch * H, T, d], k_tree, v_tree [batch * H_kv, T,
    d], caches [pages, H_kv, B, d] bf16; lengths [batch], parents [batch, T]
    int32; returns (o, lse).  Rows whose parent is -2 are not written."""
    import torch
    heads, T, d = q.shape
    batch = lengths.shape[0]
    pages, hkv = k_cache.shape[0], k_cache.shape[1]
    max_blocks = page_table.shape[-1]
    dev, h = layout.device, layout.handle
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None or lse is None:
        with _on(stream):
            o = torch.empty_like(q) if o is None else o
            lse = torch.empty((heads, T), dtype=torch.float32, device=q.device) if lse is None else lse
    rows, tree, cache = (heads, T, d), (batch * hkv, T, d), (pages, hkv, layout.B, d)
    _want(dev, torch.bfloat16, ("q", q, rows), ("k_tree", k_tree, tree), ("v_tree", v_tree, tree),
          ("k_cache", k_cache, cache), ("v_cache", v_cache, cache), ("o", o, rows))
    _want(dev, torch.int32, ("page_table", page_table, (batch, max_blocks)), ("lengths", lengths, (batch,)),
          ("parents", parents, (batch, T)))
    _want(dev, torch.float32, ("lse", lse, (heads, T)))
    workspace, size = _workspace(layout, workspace, stream, bsa_decode_tree_workspace_bytes, batch, heads, batch * hkv,
                                 T, d)
    _check(load_library().bsa_decode_tree(
        q.data_ptr(), k_tree.data_ptr(), v_tree.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        page_table.data_ptr(), max_blocks, pages, lengths.data_ptr(), parents.data_ptr(), h, T, batch, heads,
        batch * hkv, d, scale, o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), size, _stream(stream)))
    return o, lse


def bsa_get_status(layout: int, stream=None) -> None:
    _check(load_library().bsa_get_status(layout, _stream(stream)))


def bsa_debug_timeout_probe(layout: int, d: int, timeout_ns: int, stream=None) -> None:
    _check(load_library().bsa_debug_timeout_probe(layout, d, timeout_ns, _stream(stream)))


def bsa_free(layout: int) -> None:
    if layout:
        load_library().bsa_free(layout)


class Layout:
    """Owning wrapper of a layout handle (freed on ``close`` or collection)."""

    def __init__(self, kind, n, B, layout_heads=1, device=-1, **pattern):
        self.n, self.B, self.layout_heads, self.device = n, B, layout_heads, device
        self.handle = bsa_build_layout(kind, n, B, layout_heads, device, **pattern)

    @classmethod
    def for_workload(cls, w, device=-1):
        p = w.pattern
        return cls(p.kind, w.n, w.B, w.layout_heads, device, window=p.window,
                   global_first=p.global_first, dyadic_kmin=p.dyadic_kmin,
                   density=p.density, seed=p.seed)

    def csr(self):
        return bsa_layout_csr(self.handle)

    def order(self):
        return bsa_layout_order(self.handle)

    def close(self):
        if getattr(self, "handle", None):
            bsa_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def attention(q, k, v, layout: Layout, scale: float | None = None, o=None, lse=None, stream=None):
    """torch convenience: q [heads, n, d], k/v [kv_heads, n, d] bf16 CUDA tensors.

    Allocates o / lse when not given and enqueues one ``bsa_forward``.
    """
    import torch
    heads, n, d = q.shape
    kv_heads = k.shape[0]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((heads, n), dtype=torch.float32, device=q.device)
    for t in (q, k, v, o):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise BsaError(1, "q, k, v, o must be contiguous bf16 tensors")
    if lse.dtype != torch.float32 or not lse.is_contiguous():
        raise BsaError(1, "lse must be a contiguous float32 tensor")
    bsa_forward(q, k, v, layout.handle, layout.B, n, heads, kv_heads, d, scale, o, lse, stream)
    return o, lse
