"""Thin ctypes binding over libbsa.so (include/bsa.h).

Argument marshalling only: every step of the method runs in the library's
CUDA kernels.  Device tensors come from PyTorch (it provides device memory,
streams and events); work is enqueued on PyTorch's current stream.  If
libbsa.so has not been built, every call raises ``BsaError`` -- there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import numpy as np

from . import _build

BF16, FP32 = 0, 1
MASK_NONE, MASK_LOCAL_GLOBAL, MASK_SLIDING, MASK_CAUSAL = 0, 1, 2, 3
ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "parts": 3}

STATUS = {0: "BSA_OK", 1: "BSA_ERR_INVALID_ARG", 2: "BSA_ERR_UNSUPPORTED",
          3: "BSA_ERR_BAD_INDEX", 4: "BSA_ERR_WORKSPACE", 5: "BSA_ERR_CUDA",
          6: "BSA_ERR_TIMEOUT", 7: "BSA_ERR_ALIGNMENT"}

# Every symbol include/bsa.h declares.
EXPORTS = (
    "bsa_pool_blocks", "bsa_coarse_topk_workspace_size", "bsa_coarse_topk",
    "bsa_coarse_topk_ex", "bsa_fine_attention_workspace_size", "bsa_fine_attention",
    "bsa_fine_attention_lse", "bsa_fine_backward_workspace_size", "bsa_fine_backward",
    "bsa_fine_backward_lse",
    "bsa_forward_workspace_size", "bsa_forward", "bsa_forward_ex", "bsa_forward_lse",
    "bsa_forward_noalloc",
    "bsa_forward_launches", "bsa_forward_graph_create", "bsa_graph_launch", "bsa_graph_destroy",
    "bsa_static_max_blocks",
    "bsa_static_blocks", "bsa_get_device_status", "bsa_selftest_wait_timeout", "bsa_status_string",
    "bsa_last_error", "bsa_version",
    "bsa_rope_frequencies", "bsa_rope_table", "bsa_rope", "bsa_rope_backward",
    "bsa_cache_append", "bsa_cache_copy_pages", "bsa_paged_decode",
    "bsa_cache8_append", "bsa_cache8_copy_pages", "bsa_paged_decode8",
    "bsa_cache_read", "bsa_cache8_read", "bsa_paged_attention", "bsa_paged_attention8",
    "bsa_pages_create", "bsa_pages_destroy", "bsa_pages_reserve", "bsa_pages_fork",
    "bsa_pages_truncate", "bsa_pages_take_copies", "bsa_pages_compact", "bsa_pages_tables",
    "bsa_pages_free_pages",
)


class BsaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("bh", ctypes.c_int64), ("n", ctypes.c_int64),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Mask(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("window", ctypes.c_int32),
                ("stride", ctypes.c_int32), ("sliding", ctypes.c_int32)]


class ListDesc(ctypes.Structure):
    _fields_ = [("q_group", ctypes.c_int32), ("key_block", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("per_head", ctypes.c_int32)]


class Select(ctypes.Structure):
    """bsa_select: per-head budgets (device int32 [bh] or NULL), causal
    selection, always-include-local-block."""
    _fields_ = [("head_topk", ctypes.c_void_p), ("causal", ctypes.c_int32),
                ("local_block", ctypes.c_int32)]


class RopeParams(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("original", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double)]


class Heads(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("n", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Strides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("token", ctypes.c_int64)]


class Rotation(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("rot", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float)]


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("kbar", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("d", ctypes.c_int32)]


class Cache8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("kbar", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("d", ctypes.c_int32)]


class DecodeOptions(ctypes.Structure):
    _fields_ = [("local_block", ctypes.c_int32), ("share_group", ctypes.c_int32)]


class Window(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32)]


_lib = None


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libbsa.so (built in-tree); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise BsaError(5, f"{path} is missing: build it with content_dependent_block_gb300._build.build()")
    L = ctypes.CDLL(path)
    vp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                             ctypes.c_size_t, ctypes.c_float)
    sig = {
        "bsa_pool_blocks": ([Shape, vp, i32, vp, vp], i32),
        "bsa_coarse_topk_workspace_size": ([Shape, i32, i32], sz),
        "bsa_coarse_topk": ([Shape, vp, vp, i32, i32, vp, vp, sz, vp], i32),
        "bsa_coarse_topk_ex": ([Shape, vp, vp, i32, i32, ctypes.POINTER(Select), vp, vp, sz, vp],
                               i32),
        "bsa_fine_attention_workspace_size": ([Shape, ListDesc, Mask], sz),
        "bsa_fine_attention": ([Shape, vp, vp, vp, vp, ListDesc, Mask, f32, vp, vp, sz, vp], i32),
        "bsa_fine_attention_lse": ([Shape, vp, vp, vp, vp, ListDesc, Mask, f32, vp, vp, vp, sz, vp],
                                   i32),
        "bsa_fine_backward_workspace_size": ([Shape, ListDesc], sz),
        "bsa_fine_backward": ([Shape, vp, vp, vp, vp, vp, vp, ListDesc, Mask, f32, vp, vp, vp, vp, sz,
                               vp], i32),
        "bsa_fine_backward_lse": ([Shape, vp, vp, vp, vp, vp, vp, ListDesc, Mask, f32, vp, vp, vp, vp,
                                   vp, sz, vp], i32),
        "bsa_forward_workspace_size": ([Shape, i32, i32], sz),
        "bsa_forward": ([Shape, vp, vp, vp, i32, i32, f32, vp, vp, vp, sz, vp], i32),
        "bsa_forward_ex": ([Shape, vp, vp, vp, i32, i32, ctypes.POINTER(Select), f32, vp, vp, vp,
                            sz, vp], i32),
        "bsa_forward_lse": ([Shape, vp, vp, vp, i32, i32, ctypes.POINTER(Select), f32, vp, vp, vp,
                             vp, sz, vp], i32),
        "bsa_forward_noalloc": ([Shape, vp, vp, vp, i32, i32, f32, vp, vp, vp], i32),
        "bsa_forward_graph_create": ([Shape, vp, vp, vp, i32, i32, ctypes.POINTER(Select), f32, vp,
                                      vp, vp, sz, ctypes.POINTER(vp)], i32),
        "bsa_graph_launch": ([vp, vp], i32),
        "bsa_graph_destroy": ([vp], i32),
        "bsa_forward_launches": ([Shape, i32, i32], i32),
        "bsa_static_max_blocks": ([i64, i32, i32, Mask], i32),
        "bsa_static_blocks": ([i64, i32, i32, Mask, vp, i32, vp, vp], i32),
        "bsa_get_device_status": ([vp, vp], i32),
        "bsa_selftest_wait_timeout": ([i32, ctypes.c_uint64, vp], i32),
        "bsa_status_string": ([i32], ctypes.c_char_p),
        "bsa_last_error": ([], ctypes.c_char_p),
        "bsa_version": ([], i32),
        "bsa_rope_frequencies": ([RopeParams, vp], i32),
        "bsa_rope_table": ([vp, i32, vp], i32),
        "bsa_rope": ([Heads, vp, Strides, vp, i64, Rotation, vp, Strides, vp], i32),
        "bsa_rope_backward": ([Heads, vp, Strides, vp, i64, Rotation, vp, Strides, vp], i32),
        "bsa_cache_append": ([Cache, vp, i64, vp, i64, i64, i64, vp, vp, vp, i32, vp], i32),
        "bsa_cache_copy_pages": ([Cache, vp, i64, vp], i32),
        "bsa_paged_decode": ([Cache, vp, i64, i64, i32, vp, i32, i64, vp, vp, i32,
                              ctypes.POINTER(DecodeOptions), f32, vp, vp, vp], i32),
        "bsa_cache8_append": ([Cache8, vp, i64, vp, i64, i64, i64, vp, vp, vp, i32, vp], i32),
        "bsa_cache8_copy_pages": ([Cache8, vp, i64, vp], i32),
        "bsa_paged_decode8": ([Cache8, vp, i64, i64, i32, vp, i32, i64, vp, vp, i32,
                               ctypes.POINTER(DecodeOptions), f32, vp, vp, vp], i32),
        "bsa_cache_read": ([Cache, i64, i64, vp, vp, vp, i32, vp, vp, Strides, vp], i32),
        "bsa_cache8_read": ([Cache8, i64, i64, vp, vp, vp, i32, vp, vp, Strides, vp], i32),
        "bsa_paged_attention": ([Cache, vp, i64, i64, i32, vp, i32, i64, vp, vp, vp,
                                 ctypes.POINTER(Window), f32, vp, vp], i32),
        "bsa_paged_attention8": ([Cache8, vp, i64, i64, i32, vp, i32, i64, vp, vp, vp,
                                  ctypes.POINTER(Window), f32, vp, vp], i32),
        "bsa_pages_create": ([i64, i32, i32, i32, ctypes.POINTER(vp)], i32),
        "bsa_pages_destroy": ([vp], i32),
        "bsa_pages_reserve": ([vp, i32, i64], i32),
        "bsa_pages_fork": ([vp, i32, i32], i32),
        "bsa_pages_truncate": ([vp, i32, i64], i32),
        "bsa_pages_take_copies": ([vp, vp, i64, ctypes.POINTER(i64)], i32),
        "bsa_pages_compact": ([vp, vp, i64, ctypes.POINTER(i64)], i32),
        "bsa_pages_tables": ([vp, vp, vp], i32),
        "bsa_pages_free_pages": ([vp], i64),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(code: int):
    if code != 0:
        raise BsaError(code, lib().bsa_last_error().decode())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream():
    return ctypes.c_void_p(_torch().cuda.current_stream().cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _shape(t) -> Shape:
    torch = _torch()
    if t.dim() != 3 or not t.is_contiguous() or not t.is_cuda:
        raise ValueError("tensors must be contiguous CUDA [bh, n, d]")
    if t.dtype == torch.bfloat16:
        dt = BF16
    elif t.dtype == torch.float32:
        dt = FP32
    else:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return Shape(t.shape[0], t.shape[1], t.shape[2], dt)


def _workspace(nbytes: int, device):
    if nbytes == 0:
        return None
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device)


def mask_struct(kind: int = MASK_NONE, window: int = -1, stride: int = 0, sliding: int = 0) -> Mask:
    return Mask(kind, window, stride, sliding)


def pool_blocks(k, key_block: int):
    """Block means Kbar [bh, ceil(n/B), d] fp32 of bf16 keys."""
    s = _shape(k)
    nb = -(-s.n // key_block)
    kbar = _torch().empty((s.bh, nb, s.d), dtype=_torch().float32, device=k.device)
    _check(lib().bsa_pool_blocks(s, _ptr(k), key_block, _ptr(kbar), _stream()))
    return kbar


def _select(head_topk, causal: bool, local_block: bool):
    """A Select for the options, or None when there are none."""
    if head_topk is None and not causal and not local_block:
        return None
    if head_topk is not None and (head_topk.dtype != _torch().int32 or not head_topk.is_cuda
                                  or not head_topk.is_contiguous()):
        raise TypeError("head_topk must be a contiguous int32 CUDA tensor [bh]")
    return Select(None if head_topk is None else head_topk.data_ptr(), int(bool(causal)),
                  int(bool(local_block)))


def coarse_topk(q, kbar, key_block: int, topk: int, *, head_topk=None, causal: bool = False,
                local_block: bool = False):
    """Top-k block ids [bh, n, topk] int32 (ascending, -1 padded); with the
    selection options of bsa_coarse_topk_ex when any is given."""
    s = _shape(q)
    idx = _torch().empty((s.bh, s.n, topk), dtype=_torch().int32, device=q.device)
    ws_n = lib().bsa_coarse_topk_workspace_size(s, key_block, topk)
    ws = _workspace(ws_n, q.device)
    sel = _select(head_topk, causal, local_block)
    _check(lib().bsa_coarse_topk_ex(s, _ptr(q), _ptr(kbar), key_block, topk,
                                    None if sel is None else ctypes.byref(sel), _ptr(idx),
                                    _ptr(ws), ws_n, _stream()))
    return idx


def fine_attention(q, k, v, block_list=None, *, key_block: int, q_group: int = 1,
                   per_head: bool = True, mask: Optional[Mask] = None, scale: float = 0.0,
                   out=None):
    """Softmax attention of each query over its listed blocks' tokens.

    ``block_list``: int32 device tensor [bh or 1, ceil(n/q_group), max_blocks]
    (or 2-D [rows, max_blocks] when shared by all heads), None = all blocks.
    """
    s = _shape(q)
    mask = mask or mask_struct()
    if block_list is not None:
        if block_list.dtype != _torch().int32 or not block_list.is_contiguous():
            raise TypeError("block_list must be a contiguous int32 tensor")
        ld = ListDesc(q_group, key_block, block_list.shape[-1], 1 if per_head else 0)
    else:
        ld = ListDesc(1, key_block, 0, 0)
    out = _torch().empty_like(q) if out is None else out
    ws_n = lib().bsa_fine_attention_workspace_size(s, ld, mask)
    ws = _workspace(ws_n, q.device)
    _check(lib().bsa_fine_attention(s, _ptr(q), _ptr(k), _ptr(v), _ptr(block_list), ld, mask,
                                    float(scale), _ptr(out), _ptr(ws), ws_n, _stream()))
    return out


def fine_attention_lse(q, k, v, block_list, *, key_block: int, causal: bool = False,
                       scale: float = 0.0, out=None):
    """(O, lse): fine attention over the per-query lists ``block_list``
    [bh, n, k] and each query's log2-sum-exp (fp32 [bh, n]) for
    fine_backward(..., lse=lse); see bsa_fine_attention_lse in bsa.h."""
    torch = _torch()
    s = _shape(q)
    if block_list.dtype != torch.int32 or not block_list.is_contiguous():
        raise TypeError("block_list must be a contiguous int32 tensor")
    ld = ListDesc(1, key_block, block_list.shape[-1], 1)
    m = mask_struct(MASK_CAUSAL if causal else MASK_NONE)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    ws_n = lib().bsa_fine_attention_workspace_size(s, ld, m)
    ws = _workspace(ws_n, q.device)
    _check(lib().bsa_fine_attention_lse(s, _ptr(q), _ptr(k), _ptr(v), _ptr(block_list), ld, m,
                                        float(scale), _ptr(out), _ptr(lse), _ptr(ws), ws_n,
                                        _stream()))
    return out, lse


def fine_backward(q, k, v, out, dout, block_list, *, key_block: int, causal: bool = False,
                  scale: float = 0.0, lse=None):
    """Gradients (dq, dk, dv), fp32 [bh, n, d], of the fine stage over the
    per-query lists ``block_list`` [bh, n, k] (held fixed); with ``lse``
    (from fine_attention_lse on the same inputs) the softmax statistics are
    not recomputed.  See bsa_fine_backward / bsa_fine_backward_lse in bsa.h."""
    torch = _torch()
    s = _shape(q)
    if block_list.dtype != torch.int32 or not block_list.is_contiguous():
        raise TypeError("block_list must be a contiguous int32 tensor")
    ld = ListDesc(1, key_block, block_list.shape[-1], 1)
    m = mask_struct(MASK_CAUSAL if causal else MASK_NONE)
    dq, dk, dv = (torch.empty(q.shape, dtype=torch.float32, device=q.device) for _ in range(3))
    ws_n = lib().bsa_fine_backward_workspace_size(s, ld)
    ws = _workspace(ws_n, q.device)
    if lse is None:
        _check(lib().bsa_fine_backward(s, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout),
                                       _ptr(block_list), ld, m, float(scale), _ptr(dq), _ptr(dk),
                                       _ptr(dv), _ptr(ws), ws_n, _stream()))
    else:
        if lse.dtype != torch.float32 or not lse.is_contiguous():
            raise TypeError("lse must be a contiguous float32 tensor [bh, n]")
        _check(lib().bsa_fine_backward_lse(s, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout),
                                           _ptr(block_list), ld, m, float(scale), _ptr(lse),
                                           _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws_n,
                                           _stream()))
    return dq, dk, dv


class Forward:
    """Reusable forward: owns the output, selection and workspace buffers for
    one shape so repeated calls allocate nothing.  With ``graph=True`` the
    forward is captured once as a CUDA graph (bsa_forward_graph_create) for
    the q, k, v buffers of the first call and replayed with one launch; a
    call with other buffers captures again."""

    def __init__(self, bh: int, n: int, d: int, key_block: int, topk: int, device="cuda",
                 scale: float = 0.0, *, head_topk=None, causal: bool = False,
                 local_block: bool = False, graph: bool = False):
        torch = _torch()
        self.shape = Shape(bh, n, d, BF16)
        self.key_block, self.topk, self.scale = key_block, topk, scale
        self.head_topk = head_topk            # kept alive: the library reads it on every call
        self.sel = _select(head_topk, causal, local_block)
        self.use_graph = graph
        self._graph = None                    # (handle, (q, k, v) pointers, keep_idx)
        self.ws_bytes = lib().bsa_forward_workspace_size(self.shape, key_block, topk)
        self.ws = _workspace(self.ws_bytes, device)
        self.out = torch.empty((bh, n, d), dtype=torch.bfloat16, device=device)
        self.idx = torch.empty((bh, n, topk), dtype=torch.int32, device=device)

    @property
    def launches(self) -> int:
        """Kernel launches one call enqueues."""
        return int(lib().bsa_forward_launches(self.shape, self.key_block, self.topk))

    def __call__(self, q, k, v, keep_idx: bool = True):
        s = _shape(q)
        if (s.bh, s.n, s.d) != (self.shape.bh, self.shape.n, self.shape.d):
            raise ValueError("shape differs from the one this Forward was built for")
        sel = None if self.sel is None else ctypes.byref(self.sel)
        if not self.use_graph:
            _check(lib().bsa_forward_ex(self.shape, _ptr(q), _ptr(k), _ptr(v), self.key_block,
                                        self.topk, sel, float(self.scale), _ptr(self.out),
                                        _ptr(self.idx if keep_idx else None), _ptr(self.ws),
                                        self.ws_bytes, _stream()))
            return self.out
        key = ((q.data_ptr(), k.data_ptr(), v.data_ptr()), keep_idx)
        if self._graph is None or self._graph[1] != key:
            self.close()
            h = ctypes.c_void_p()
            _check(lib().bsa_forward_graph_create(
                self.shape, _ptr(q), _ptr(k), _ptr(v), self.key_block, self.topk, sel,
                float(self.scale), _ptr(self.out), _ptr(self.idx if keep_idx else None),
                _ptr(self.ws), self.ws_bytes, ctypes.byref(h)))
            self._graph = (h, key)
        _check(lib().bsa_graph_launch(self._graph[0], _stream()))
        return self.out

    def close(self):
        """Release the captured graph, if any."""
        if self._graph is not None:
            lib().bsa_graph_destroy(self._graph[0])
            self._graph = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def forward(q, k, v, key_block: int, topk: int, scale: float = 0.0, *, head_topk=None,
            causal: bool = False, local_block: bool = False) -> Tuple[object, object]:
    """Whole dynamic forward (with the selection options of bsa_forward_ex);
    returns (out, idx)."""
    s = _shape(q)
    f = Forward(s.bh, s.n, s.d, key_block, topk, device=q.device, scale=scale,
                head_topk=head_topk, causal=causal, local_block=local_block)
    out = f(q, k, v, keep_idx=True)
    return out, f.idx


def forward_lse(q, k, v, key_block: int, topk: int, scale: float = 0.0, *, head_topk=None,
                causal: bool = False, local_block: bool = False):
    """Whole dynamic forward that also keeps each query's log2-sum-exp for
    fine_backward(..., lse=lse); returns (out, idx, lse).  See
    bsa_forward_lse in bsa.h."""
    torch = _torch()
    s = _shape(q)
    out = torch.empty_like(q)
    idx = torch.empty((s.bh, s.n, topk), dtype=torch.int32, device=q.device)
    lse = torch.empty((s.bh, s.n), dtype=torch.float32, device=q.device)
    sel = _select(head_topk, causal, local_block)
    ws_n = lib().bsa_forward_workspace_size(s, key_block, topk)
    ws = _workspace(ws_n, q.device)
    _check(lib().bsa_forward_lse(s, _ptr(q), _ptr(k), _ptr(v), key_block, topk,
                                 None if sel is None else ctypes.byref(sel), float(scale),
                                 _ptr(out), _ptr(idx), _ptr(lse), _ptr(ws), ws_n, _stream()))
    return out, idx, lse


def forward_noalloc(q, k, v, key_block: int, topk: int, scale: float = 0.0, out=None, idx=None):
    """Whole dynamic forward using the library's static scratch (no workspace
    allocation); returns (out, idx).  See bsa_forward_noalloc in bsa.h."""
    torch = _torch()
    s = _shape(q)
    out = torch.empty_like(q) if out is None else out
    idx = torch.empty((s.bh, s.n, topk), dtype=torch.int32, device=q.device) if idx is None else idx
    _check(lib().bsa_forward_noalloc(s, _ptr(q), _ptr(k), _ptr(v), key_block, topk, float(scale),
                                     _ptr(out), _ptr(idx), _stream()))
    return out, idx


def static_blocks(n: int, q_group: int, key_block: int, mask: Mask):
    """Host-built static list: (list [rows, max_blocks] int32, counts, active_pairs)."""
    L = lib()
    mb = L.bsa_static_max_blocks(n, q_group, key_block, mask)
    if mb < 0:
        raise BsaError(-mb, L.bsa_last_error().decode() or "bad static-list arguments")
    rows = -(-n // q_group)
    lst = np.empty((rows, max(mb, 1)), dtype=np.int32)
    counts = np.empty(rows, dtype=np.int32)
    pairs = ctypes.c_int64(0)
    _check(L.bsa_static_blocks(n, q_group, key_block, mask,
                               lst.ctypes.data_as(ctypes.c_void_p), lst.shape[1],
                               counts.ctypes.data_as(ctypes.c_void_p), ctypes.byref(pairs)))
    return lst, counts, int(pairs.value)


def device_status() -> int:
    """Read and clear the device status word (synchronises the stream)."""
    v = ctypes.c_int32(0)
    _check(lib().bsa_get_device_status(ctypes.byref(v), _stream()))
    return int(v.value)


def selftest_wait_timeout(kind: int, limit_ns: int) -> None:
    """Enqueue the bounded-wait self-test (bsa_selftest_wait_timeout): a wait
    nothing completes gives up after about limit_ns and records
    BSA_ERR_TIMEOUT; read it with device_status()."""
    _check(lib().bsa_selftest_wait_timeout(int(kind), int(limit_ns), _stream()))


def _whole(x, bits: int, name: str) -> int:
    """x as an integer of `bits` bits; ctypes would keep the low ones of any."""
    i = int(x)
    if i != x or not -(1 << (bits - 1)) <= i < 1 << (bits - 1):
        raise ValueError(f"{name} must be a whole number of {bits} bits (got {x})")
    return i


# ------------------------------------------------------------ rotary positions
class Rope:
    """A rotation's plan: frequencies, fixed-point table on the device, layout
    and factor (see bsa_rope_params and bsa_rotation in bsa.h).  ``inv_freq``
    replaces the computed frequencies by the caller's (rot / 2 numbers)."""

    def __init__(self, rot: int, theta: float = 10000.0, *, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original: float = 0.0,
                 low: float = 1.0, high: float = 32.0, attention_factor: float = 1.0,
                 inv_freq=None, device="cuda"):
        torch = _torch()
        rot = _whole(rot, 32, "rot")
        if inv_freq is None:
            p = RopeParams(rot, ROPE_SCALING[scaling], theta, factor, original, low, high)
            self.inv_freq = np.empty(max(rot, 2) // 2, dtype=np.float64)
            _check(lib().bsa_rope_frequencies(p, self.inv_freq.ctypes.data_as(ctypes.c_void_p)))
        else:
            self.inv_freq = np.ascontiguousarray(inv_freq, dtype=np.float64)
            if self.inv_freq.shape != (rot // 2,) or rot % 2:
                raise ValueError("inv_freq must hold rot / 2 numbers")
        table = np.empty(self.inv_freq.shape, dtype=np.uint64)
        _check(lib().bsa_rope_table(self.inv_freq.ctypes.data_as(ctypes.c_void_p), table.size,
                                    table.ctypes.data_as(ctypes.c_void_p)))
        self.rot, self.interleaved, self.attention_factor = rot, interleaved, attention_factor
        self.table = torch.from_numpy(table.view(np.int64)).to(device)
        self.rotation = Rotation(self.table.data_ptr(), rot, int(interleaved), attention_factor)


# The calls below cost some microseconds on the host against some on the
# device, so their checks read each attribute once.
def _here(*tensors) -> int:
    """The current device's stream, all tensors being on that device: pointers
    of another one would be launched on this one's stream."""
    C = _torch()._C
    here = C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError("tensors must be on the current CUDA device")
    return C._cuda_getCurrentRawStream(here)


def _written(*tensors):
    """A tensor of the caller's is written through its pointer: autograd, which
    does not see that, is to refuse what it saved of it."""
    _torch_module.autograd.graph.increment_version(tensors)


def _i32(t, name: str, shape):
    if t.shape != shape or t.dtype is not _torch_module.int32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor {list(shape)}")
    return t.data_ptr()


def _rope(fn, x, rope: Rope, positions, out):
    torch = _torch()
    shape, dtype, xs = x.shape, x.dtype, x.stride()
    dims = len(shape)
    if dims not in (3, 4) or xs[-1] != 1:
        raise ValueError("x must be [batch, heads, n, d] or [heads, n, d] with contiguous channels")
    if dtype is torch.bfloat16:
        dt = BF16
    elif dtype is torch.float32:
        dt = FP32
    else:
        raise TypeError(f"unsupported dtype {dtype}")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.shape != shape or out.dtype is not dtype or out.stride(-1) != 1:
        raise ValueError("out must have x's shape and dtype and contiguous channels")
    if torch.is_grad_enabled() and (x.requires_grad or out.requires_grad):
        raise ValueError("rope and rope_backward record no history: call them under no_grad or in "
                         "the forward and backward of an autograd function")
    os_ = out.stride()
    if dims == 4:
        batch, heads, n, d = shape
        xs, os_ = Strides(xs[0], xs[1], xs[2]), Strides(os_[0], os_[1], os_[2])
    else:
        batch, (heads, n, d) = 1, shape
        xs, os_ = Strides(0, xs[0], xs[1]), Strides(0, os_[0], os_[1])
    if isinstance(positions, torch.Tensor):
        if positions.dim() == 2:
            pos = _i32(positions, "positions", (batch, n))
        elif batch == 1:
            pos = _i32(positions, "positions", (n,))
        else:
            raise TypeError("positions must be [batch, n]")
        first, stream = 0, _here(x, out, rope.table, positions)
    else:
        first, pos, stream = _whole(positions, 64, "positions"), None, _here(x, out, rope.table)
    _check(fn(Heads(batch, n, heads, d, dt), x.data_ptr(), xs, pos, first, rope.rotation,
              out.data_ptr(), os_, stream))
    _written(out)
    return out


def rope(x, rope: Rope, positions=0, *, out=None):
    """Rotated x: [batch, heads, n, d] (or [heads, n, d]), any strides with
    contiguous channels.  ``positions``: the first token's position, or an
    int32 device tensor [batch, n].  ``out`` may be x itself; by default a
    contiguous tensor, the layout ``forward`` takes.  Autograd does not record
    it: ``rope_backward`` is its gradient."""
    return _rope(lib().bsa_rope, x, rope, positions, out)


def rope_backward(dout, rope: Rope, positions=0, *, out=None):
    """Gradient of ``rope`` with respect to its input."""
    return _rope(lib().bsa_rope_backward, dout, rope, positions, out)


# ---------------------------------------------------------------- paged cache
class PagedCache:
    """A paged cache's device tensors: k, v [pages, heads, page, d] bf16 and
    the block means kbar [pages, heads, d] fp32 (bsa_cache in bsa.h)."""
    _calls = ("bsa_cache_append", "bsa_cache_copy_pages", "bsa_paged_decode", "bsa_cache_read",
              "bsa_paged_attention")

    def __init__(self, k, v, kbar):
        torch = _torch()
        if k.dim() != 4 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16 \
                or k.shape != v.shape or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous bfloat16 [pages, heads, page, d]")
        _check_means(kbar, k.shape)
        _here(k, v, kbar)
        self.k, self.v, self.kbar = k, v, kbar
        self.num_pages, self.heads, self.page, self.d = k.shape
        self.struct = Cache(k.data_ptr(), v.data_ptr(), kbar.data_ptr(), self.num_pages,
                            self.heads, self.page, self.d)
        self._bind(k, v, kbar)

    def _bind(self, *written):
        """The tensors that appends and copies write, and the entry points for
        this kind of cache."""
        self.written = written
        self._append, self._copy, self._decode, self._read, self._attention = \
            (getattr(lib(), name) for name in self._calls)

    @classmethod
    def empty(cls, num_pages: int, heads: int, page: int, d: int, device="cuda"):
        torch = _torch()
        k, v = (torch.zeros((num_pages, heads, page, d), dtype=torch.bfloat16, device=device)
                for _ in range(2))
        return cls(k, v, torch.zeros((num_pages, heads, d), dtype=torch.float32, device=device))


def _check_means(kbar, shape):
    if kbar.dtype != _torch().float32 or not kbar.is_contiguous() \
            or tuple(kbar.shape) != (shape[0], shape[1], shape[3]):
        raise ValueError("kbar must be contiguous float32 [pages, heads, d]")


class PagedCache8(PagedCache):
    """A paged cache in 8 bits: k, v [pages, heads, page, d] int8, k_scale,
    v_scale [pages, heads, page] fp32 and the block means kbar [pages, heads,
    d] fp32 (bsa_cache8 in bsa.h).  A row stands for its codes times its
    scale; ``cache_append`` quantises bf16 rows.  Every function that takes a
    PagedCache takes either kind."""
    _calls = ("bsa_cache8_append", "bsa_cache8_copy_pages", "bsa_paged_decode8", "bsa_cache8_read",
              "bsa_paged_attention8")

    def __init__(self, k, v, k_scale, v_scale, kbar):
        torch = _torch()
        if k.dim() != 4 or k.dtype != torch.int8 or v.dtype != torch.int8 \
                or k.shape != v.shape or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous int8 [pages, heads, page, d]")
        for scale in (k_scale, v_scale):
            if scale.dtype != torch.float32 or not scale.is_contiguous() or scale.shape != k.shape[:3]:
                raise ValueError("k_scale and v_scale must be contiguous float32 [pages, heads, page]")
        _check_means(kbar, k.shape)
        _here(k, v, k_scale, v_scale, kbar)
        self.k, self.v, self.k_scale, self.v_scale, self.kbar = k, v, k_scale, v_scale, kbar
        self.num_pages, self.heads, self.page, self.d = k.shape
        self.struct = Cache8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                             kbar.data_ptr(), self.num_pages, self.heads, self.page, self.d)
        self._bind(k, v, k_scale, v_scale, kbar)

    @classmethod
    def empty(cls, num_pages: int, heads: int, page: int, d: int, device="cuda"):
        torch = _torch()
        k, v = (torch.zeros((num_pages, heads, page, d), dtype=torch.int8, device=device)
                for _ in range(2))
        ks, vs = (torch.zeros((num_pages, heads, page), dtype=torch.float32, device=device)
                  for _ in range(2))
        return cls(k, v, ks, vs, torch.zeros((num_pages, heads, d), dtype=torch.float32, device=device))


def _token_rows(t, name: str, heads: int, d: int) -> int:
    """The stride from a token's rows to the next's."""
    shape, strides = t.shape, t.stride()
    if shape[1:] != (heads, d) or t.dtype is not _torch().bfloat16 or strides[2] != 1 \
            or (heads > 1 and strides[1] != d):
        raise ValueError(f"{name} must be bfloat16 [tokens, {heads}, {d}] with contiguous rows")
    return strides[0] if shape[0] > 1 else heads * d


def cache_append(cache: PagedCache, k, v, table, start, *, cu_tokens=None):
    """Append k, v [tokens, heads, d] (token stride free) to their sequences'
    pages and refresh the touched blocks' means.  ``table`` int32 [seqs,
    width], ``start`` int32 [seqs] (lengths before); ``cu_tokens`` int32
    [seqs + 1], None: as many tokens for each.  See bsa_cache_append."""
    seqs, width = table.shape
    ks = _token_rows(k, "k", cache.heads, cache.d)
    vs = _token_rows(v, "v", cache.heads, cache.d)
    if k.shape != v.shape:
        raise ValueError("k and v must have one shape")
    cu = None if cu_tokens is None else _i32(cu_tokens, "cu_tokens", (seqs + 1,))
    _check(cache._append(
        cache.struct, k.data_ptr(), ks, v.data_ptr(), vs, k.shape[0], seqs, cu,
        _i32(start, "start", (seqs,)), _i32(table, "table", (seqs, width)), width,
        _here(cache.k, k, v, table, start, cu_tokens)))
    _written(*cache.written)


def copy_pages(cache: PagedCache, pairs):
    """Copy whole pages: ``pairs`` int32 [count, 2] of (from, to) on the
    device, or a host array as PageTable hands them out."""
    torch = _torch()
    if not isinstance(pairs, torch.Tensor):
        pairs = np.asarray(pairs).reshape(-1, 2)
        if len(np.unique(pairs[:, 1])) < len(pairs) or np.isin(pairs[:, 1], pairs[:, 0]).any():
            raise ValueError("a page is the target of two pairs, or of one and the source of another")
        if pairs.size and not (np.abs(pairs) < 1 << 31).all() or (pairs != np.floor(pairs)).any():
            raise ValueError("pairs must be whole numbers of 32 bits")
        pairs = torch.from_numpy(np.ascontiguousarray(pairs, dtype=np.int32)).to(cache.k.device)
    count = pairs.shape[0]
    _check(cache._copy(cache.struct, _i32(pairs, "pairs", (count, 2)), count,
                       _here(cache.k, pairs)))
    _written(*cache.written)


_OPTIONS = {(local, share): ctypes.byref(DecodeOptions(local, share))
            for local in (False, True) for share in (False, True)}


def paged_decode(cache: PagedCache, q, table, lens, topk: int, *, token_seq=None,
                 local_block: bool = True, share_group: bool = False, scale: float = 0.0,
                 out=None):
    """(out, idx): each token of q [tokens, q_heads, d] attends to the first
    ``lens`` keys of its sequence, in the topk blocks it selects.  idx int32
    [tokens, q_heads or cache heads, topk], ascending, -1 padded.  See
    bsa_paged_decode in bsa.h."""
    torch = _torch()
    seqs, width = table.shape
    tokens, q_heads, d = q.shape
    qs = _token_rows(q, "q", q_heads, cache.d)
    seq = None if token_seq is None else _i32(token_seq, "token_seq", (tokens,))
    if out is None:
        out = torch.empty((tokens, q_heads, d), dtype=q.dtype, device=q.device)
    elif out.dtype is not q.dtype or out.shape != (tokens, q_heads, d) or not out.is_contiguous():
        raise ValueError("out must be contiguous bfloat16 [tokens, q_heads, d]")
    idx = torch.empty((tokens, cache.heads if share_group else q_heads, topk), dtype=torch.int32,
                      device=q.device)
    _check(cache._decode(
        cache.struct, q.data_ptr(), qs, tokens, q_heads, _i32(table, "table", (seqs, width)), width,
        seqs, seq, _i32(lens, "lens", (tokens,)), topk,
        _OPTIONS[bool(local_block), bool(share_group)], scale, out.data_ptr(),
        idx.data_ptr(), _here(cache.k, q, table, lens, token_seq, out)))
    _written(out)
    return out, idx


def cache_read(cache: PagedCache, table, start, tokens: int, *, cu_tokens=None,
               heads_first: bool = False, out=None):
    """(k, v) bf16 of cached tokens: sequence s's positions from ``start`` on,
    ``tokens`` in all, cut by ``cu_tokens`` (None: as many for each), as
    [tokens, heads, d], or [heads, tokens, d] with ``heads_first`` (the layout
    ``forward`` takes).  ``out``: a pair of tensors of that shape, of one
    layout, with contiguous channels.  Rows of tokens that no sequence has are
    not written.  See bsa_cache_read in bsa.h."""
    torch = _torch()
    seqs, width = table.shape
    heads, d = cache.heads, cache.d
    if type(tokens) is not int:
        tokens = _whole(tokens, 64, "tokens")
    shape = (heads, tokens, d) if heads_first else (tokens, heads, d)
    if out is None:
        k = torch.empty(shape, dtype=torch.bfloat16, device=cache.k.device)
        v = torch.empty_like(k)
        st = (shape[1] * d, d)
    else:
        k, v = out
        for t in out:
            if t.shape != shape or t.dtype is not torch.bfloat16 or t.stride(2) != 1:
                raise ValueError(f"out must be two bfloat16 {list(shape)} with contiguous channels")
        st = k.stride()
        if v.stride() != st:
            raise ValueError("out's tensors must have one layout")
        if torch.is_grad_enabled() and (k.requires_grad or v.requires_grad):
            raise ValueError("cache_read records no history: out must not require a gradient")
    cu = None if cu_tokens is None else _i32(cu_tokens, "cu_tokens", (seqs + 1,))
    _check(cache._read(
        cache.struct, tokens, seqs, cu, _i32(start, "start", (seqs,)),
        _i32(table, "table", (seqs, width)), width, k.data_ptr(), v.data_ptr(),
        Strides(0, st[0], st[1]) if heads_first else Strides(0, st[1], st[0]),
        _here(cache.k, table, start, cu_tokens, k, v)))
    if out is not None:
        _written(k, v)
    return k, v


def _window(window, sinks):
    """A reference to the bsa_window of these numbers, None for none."""
    # what is kept goes by the values: a tensor or array may change in place
    if type(window) is not int or type(sinks) is not int:
        window, sinks = _whole(window, 32, "window"), _whole(sinks, 32, "sinks")
    return _window_of(window, sinks)


@functools.lru_cache(maxsize=64)
def _window_of(window: int, sinks: int):
    window, sinks = _whole(window, 32, "window"), _whole(sinks, 32, "sinks")
    if window == 0 and sinks != 0:
        raise ValueError("sinks without a window")
    return None if window == 0 else ctypes.byref(Window(window, sinks))


def paged_attention(cache: PagedCache, q, table, start, *, cu_tokens=None, tree=None,
                    window: int = 0, sinks: int = 0, scale: float = 0.0, out=None):
    """Attention of new tokens q [tokens, q_heads, d], whose K and V the cache
    holds from position ``start`` of each sequence on, to all keys up to
    themselves.  ``cu_tokens`` int32 [seqs + 1], None: as many tokens for each.
    ``tree`` int64 [tokens]: which of its sequence's (at most 64) new tokens a
    token sees, besides the prefix.  ``window`` W and ``sinks``: only the last W
    positions and the first few; 0: all.  Rows of tokens that no sequence has are
    not written.  See bsa_paged_attention in bsa.h."""
    torch = _torch()
    seqs, width = table.shape
    tokens, q_heads, d = q.shape
    qs = _token_rows(q, "q", q_heads, cache.d)
    cu = None if cu_tokens is None else _i32(cu_tokens, "cu_tokens", (seqs + 1,))
    if tree is not None and (tree.shape != (tokens,) or tree.dtype is not torch.int64
                             or not tree.is_contiguous()):
        raise TypeError(f"tree must be a contiguous int64 tensor {[tokens]}")
    span, fresh = _window(window, sinks), out is None
    if fresh:
        out = torch.empty((tokens, q_heads, d), dtype=q.dtype, device=q.device)
    elif out.dtype is not q.dtype or out.shape != (tokens, q_heads, d) or not out.is_contiguous():
        raise ValueError("out must be contiguous bfloat16 [tokens, q_heads, d]")
    if torch.is_grad_enabled() and (q.requires_grad or out.requires_grad):
        raise ValueError("paged_attention records no history: call it under no_grad")
    _check(cache._attention(
        cache.struct, q.data_ptr(), qs, tokens, q_heads, _i32(table, "table", (seqs, width)), width,
        seqs, cu, _i32(start, "start", (seqs,)), None if tree is None else tree.data_ptr(),
        span, scale, out.data_ptr(), _here(cache.k, q, table, start, cu_tokens, tree, out)))
    if not fresh:
        _written(out)
    return out


class PageTable:
    """Which sequence owns which page (host side, bsa_pages_* in bsa.h):
    ``reserve`` room, ``fork`` with copy on write, ``truncate`` or ``free``,
    ``compact``.  ``take_copies`` and ``compact`` return int32 [count, 2]
    arrays for ``copy_pages``; run the former's before the next append.
    A step reserves, runs the copies, and appends what it reserved; fork
    before the reserves or after the append (``take_copies`` refuses copies
    that would miss tokens, see bsa_pages_take_copies in bsa.h)."""

    def __init__(self, num_pages: int, page: int, max_seqs: int, width: int):
        self._h = ctypes.c_void_p()
        num_pages, page = _whole(num_pages, 64, "num_pages"), _whole(page, 32, "page")
        max_seqs, width = _whole(max_seqs, 32, "max_seqs"), _whole(width, 32, "width")
        self.num_pages, self.max_seqs, self.width = num_pages, max_seqs, width
        _check(lib().bsa_pages_create(num_pages, page, max_seqs, width, ctypes.byref(self._h)))

    def reserve(self, seq: int, tokens: int):
        _check(lib().bsa_pages_reserve(self._h, _whole(seq, 32, "seq"), _whole(tokens, 64, "tokens")))

    def fork(self, source: int, to: int):
        _check(lib().bsa_pages_fork(self._h, _whole(source, 32, "source"), _whole(to, 32, "to")))

    def truncate(self, seq: int, length: int):
        _check(lib().bsa_pages_truncate(self._h, _whole(seq, 32, "seq"), _whole(length, 64, "length")))

    def free(self, seq: int):
        self.truncate(seq, 0)

    def _pairs(self, fn):
        count = ctypes.c_int64(0)
        _check(fn(self._h, None, 0, ctypes.byref(count)))
        pairs = np.empty((count.value, 2), dtype=np.int32)
        _check(fn(self._h, pairs.ctypes.data_as(ctypes.c_void_p), count.value,
                  ctypes.byref(count)))
        return pairs

    def take_copies(self):
        return self._pairs(lib().bsa_pages_take_copies)

    def compact(self):
        return self._pairs(lib().bsa_pages_compact)

    def tables(self):
        """(table int32 [max_seqs, width], lengths int32 [max_seqs])."""
        table = np.empty((self.max_seqs, self.width), dtype=np.int32)
        lengths = np.empty(self.max_seqs, dtype=np.int32)
        _check(lib().bsa_pages_tables(self._h, table.ctypes.data_as(ctypes.c_void_p),
                                      lengths.ctypes.data_as(ctypes.c_void_p)))
        return table, lengths

    @property
    def free_pages(self) -> int:
        return int(lib().bsa_pages_free_pages(self._h))

    def close(self):
        if self._h:
            lib().bsa_pages_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
