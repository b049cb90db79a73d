"""Paged key/value cache and attention of new tokens over it.

A cache is ``k_pages`` and ``v_pages`` [pages, H, page_size, 128], BF16, or
E4M3 (``torch.float8_e4m3fn``) with one power-of-two scale a row, held as
exponent bytes ``k_exp`` and ``v_exp`` (uint8 [pages, H, page_size]: e stands
for 2^(e - 127)).  A batch is three int32 CUDA tensors: ``table``
[sequences, width] (the pages of each sequence in order), ``row_start``
[sequences + 1] (the rows of each sequence in a packed tensor) and ``kv_len``
[sequences] (its cached tokens, the new ones among them).  The n rows of a
sequence are its last n tokens.  ``include/sparse_attn.h`` states the format,
what a call does for positions below 0, and what is checked on the device.

* ``cache_write``: rows of K and V into the cache;
* ``cache_read``: the inverse, the packed BF16 tensors of ``sparse_attn``;
* ``paged_attn``: attention of rows of Q over the cache, for chunks of new
  tokens and for single ones.

Nothing here waits for the GPU.  With ``ws`` (a workspace of
``paged_workspace``, or 256 bytes for the two copies)
``sparse_attn_last_device_status(ws)`` tells what the device found wrong.
"""

from __future__ import annotations

import ctypes
import functools
import math

from . import _native
from ._native import SA_OK, SaPagedParams, SparseAttnError

PAGE_SIZES = (16, 32, 64, 128)


def _torch():
    import torch

    return torch


def paged_cache(pages, H, page_size=64, dtype="bf16", device="cuda"):
    """An uninitialised cache: (k_pages, v_pages, k_exp, v_exp); the exponents
    are None for ``dtype`` "bf16" and tensors for "e4m3"."""
    torch = _torch()
    kinds = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
    if dtype not in kinds:
        raise ValueError("dtype must be 'bf16' or 'e4m3'")
    if page_size not in PAGE_SIZES:
        raise ValueError(f"page_size must be one of {PAGE_SIZES}")
    shape = (pages, H, page_size, 128)
    k, v = (torch.empty(shape, dtype=kinds[dtype], device=device) for _ in range(2))
    if dtype == "bf16":
        return k, v, None, None
    ke, ve = (torch.empty(shape[:3], dtype=torch.uint8, device=device) for _ in range(2))
    return k, v, ke, ve


@functools.lru_cache(maxsize=4096)
def _params(pages_shape, kind, table_shape, table_stride, rows, max_new, Hq, causal, window, scale, strides):
    """The C parameters of a call's sizes (a plain function of numbers)."""
    return SaPagedParams(_native.SA_ABI_VERSION, kind, pages_shape[0], pages_shape[1], pages_shape[2],
                         pages_shape[3], table_shape[0], table_shape[1], table_stride, rows, max_new, Hq, causal,
                         window, scale, *strides)


def _check(cond, text):
    if not cond:
        raise ValueError(text)


def _cache(k_pages, v_pages, k_exp, v_exp):
    """Checks the cache's tensors; returns (kind, shape, device index)."""
    torch = _torch()
    shape, dtype = k_pages.shape, k_pages.dtype
    if dtype is torch.bfloat16:
        kind = _native.SA_CACHE_BF16
    elif dtype is torch.float8_e4m3fn:
        kind = _native.SA_CACHE_E4M3
    else:
        raise TypeError("k_pages must be bfloat16 or float8_e4m3fn")
    if v_pages.dtype is not dtype:
        raise TypeError("k_pages and v_pages must have the same dtype")
    dev = k_pages.get_device()
    _check(dev >= 0, "k_pages must be a CUDA tensor")
    _check(len(shape) == 4 and v_pages.shape == shape, "k_pages and v_pages must be [pages, H, page_size, 128]")
    _check(k_pages.is_contiguous() and v_pages.is_contiguous(), "k_pages and v_pages must be contiguous")
    _check(v_pages.get_device() == dev, "v_pages must be on k_pages' device")
    if kind == _native.SA_CACHE_E4M3:
        for t, n in ((k_exp, "k_exp"), (v_exp, "v_exp")):
            if t is None or t.dtype is not torch.uint8 or t.shape != shape[:3] or not t.is_contiguous() \
                    or t.get_device() != dev:
                raise ValueError(f"{n}: contiguous uint8 [pages, H, page_size] on the cache's device required")
    elif k_exp is not None or v_exp is not None:
        raise ValueError("a bfloat16 cache has no exponents")
    return kind, shape, dev


def _batch(table, row_start, kv_len, dev):
    i32 = _torch().int32
    for t, n in ((table, "table"), (row_start, "row_start"), (kv_len, "kv_len")):
        if t.dtype is not i32 or t.get_device() != dev:
            raise ValueError(f"{n} must be an int32 tensor on the cache's device")
    _check(table.dim() == 2 and (table.shape[1] < 2 or table.stride(1) == 1),
           "table must be [sequences, width] with contiguous rows")
    n = table.shape[0]
    _check(row_start.shape == (n + 1,) and row_start.is_contiguous(), "row_start must be contiguous [sequences + 1]")
    _check(kv_len.shape == (n,) and kv_len.is_contiguous(), "kv_len must be contiguous [sequences]")


def _rows(t, name, heads, dev):
    """Rows [n, heads, 128] (or [1, n, heads, 128]); returns (rows, token stride, head stride)."""
    if t.dtype is not _torch().bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    shape, stride = t.shape, t.stride()
    if len(shape) == 4 and shape[0] == 1:
        shape, stride = shape[1:], stride[1:]
    _check(len(shape) == 3 and shape[2] == 128 and (heads is None or shape[1] == heads),
           f"{name} must be [rows, heads, 128], got {tuple(t.shape)}")
    _check(t.get_device() == dev, f"{name} must be on the cache's device")
    n, h = shape[0], shape[1]
    # strides of dimensions of one element mean nothing
    ts, hs = (stride[0] if n > 1 else 0), (stride[1] if h > 1 else 0)
    _check(stride[2] == 1 and ts % 8 == 0 and hs % 8 == 0,
           f"{name}: contiguous last dimension and strides that are multiples of 8 required")
    return n, ts, hs


def _out(t, name, shape, dtype, dev):
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev)), True
    if t.dtype is not dtype or not t.is_contiguous() or t.numel() != math.prod(shape) or t.get_device() != dev:
        raise ValueError(f"{name}: contiguous {dtype} {tuple(shape)} on the cache's device required")
    return t, False


def _scratch(ws, dev):
    if ws.dtype is not _torch().uint8 or not ws.is_contiguous() or ws.get_device() != dev:
        raise ValueError("ws must be a contiguous uint8 tensor on the cache's device")
    return ws.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name, dev, stream, fresh, *args):
    """Runs a C entry point on ``stream`` (default: the device's current one).
    ``fresh``: tensors allocated here, kept for the stream that uses them."""
    torch = _torch()
    here = torch.cuda.current_stream(dev)
    if stream is None:
        stream = here
    elif stream != here:
        for t in fresh:
            t.record_stream(stream)
    fn = getattr(_native.load_library(), name)
    if torch.cuda.current_device() == dev:
        st = fn(*args, stream.cuda_stream or None)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream.cuda_stream or None)
    if st != SA_OK:
        raise SparseAttnError(st, name)


def cache_write(k, v, k_pages, v_pages, table, row_start, kv_len, k_exp=None, v_exp=None, ws=None, stream=None):
    """Writes the rows of k and v (bf16 [rows, H, 128], any strides that are
    multiples of 8) to their sequences' pages, quantised for an E4M3 cache."""
    kind, shape, dev = _cache(k_pages, v_pages, k_exp, v_exp)
    _batch(table, row_start, kv_len, dev)
    n, kt, kh = _rows(k, "k", shape[1], dev)
    nv, vt, vh = _rows(v, "v", shape[1], dev)
    _check(n == nv, "k and v must have the same rows")
    p = _params(shape, kind, table.shape, table.stride(0), n, n, shape[1], 1, 0, 1.0, (kt, kh, vt, vh))
    _call("sparse_attn_cache_write", dev, stream, (), ctypes.byref(p), k.data_ptr(), v.data_ptr(),
          k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_exp), _ptr(v_exp), table.data_ptr(), row_start.data_ptr(),
          kv_len.data_ptr(), None if ws is None else _scratch(_ws256(ws), dev))


def _ws256(ws):
    _check(ws.numel() >= 256, "ws must have 256 bytes at least")
    return ws


def cache_read(k_pages, v_pages, table, row_start, kv_len, rows=None, k_exp=None, v_exp=None, k=None, v=None, ws=None,
               stream=None):
    """The rows of every sequence as bf16 (k, v) [rows, H, 128].  ``rows`` (the
    last row_start) sizes the outputs when k and v are not given."""
    torch = _torch()
    kind, shape, dev = _cache(k_pages, v_pages, k_exp, v_exp)
    _batch(table, row_start, kv_len, dev)
    if rows is None:
        _check(k is not None, "give rows, or k and v")
        rows = _rows(k, "k", shape[1], dev)[0]
    out = (rows, shape[1], 128)
    k, fk = _out(k, "k", out, torch.bfloat16, dev)
    v, fv = _out(v, "v", out, torch.bfloat16, dev)
    p = _params(shape, kind, table.shape, table.stride(0), rows, rows, shape[1], 1, 0, 1.0, (0, 0, 0, 0))
    _call("sparse_attn_cache_read", dev, stream, [t for t, f in ((k, fk), (v, fv)) if f], ctypes.byref(p),
          k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_exp), _ptr(v_exp), table.data_ptr(), row_start.data_ptr(),
          kv_len.data_ptr(), k.data_ptr(), v.data_ptr(), None if ws is None else _scratch(_ws256(ws), dev))
    return k, v


def _attn_params(q, kind, shape, table, max_new, causal, window, scale, dev):
    n, qt, qh = _rows(q, "q", None, dev)
    hq = q.shape[-2]
    _check(hq % shape[1] == 0 and hq > 0, "q's heads must be a multiple of the cache's")
    _check(window >= 0 and (causal or window == 0), "window: 0, or a positive number with causal=True")
    max_new = n if max_new is None else min(int(max_new), n)
    _check(max_new >= 0, "max_new must not be negative")
    scale = 1.0 / math.sqrt(128.0) if scale is None else float(scale)
    return n, hq, _params(shape, kind, table.shape, table.stride(0), n, max_new, hq, 1 if causal else 0, int(window),
                          scale, (qt, qh, 0, 0))


def paged_workspace(q, k_pages, table, max_new=None):
    """A workspace for ``paged_attn`` calls of these sizes.  It belongs to one
    stream at a time; two captured graphs that may run at once need two."""
    torch = _torch()
    dev = k_pages.get_device()
    return torch.empty(paged_ws_bytes(q, k_pages, table, max_new), dtype=torch.uint8,
                       device=torch.device("cuda", dev))


def paged_ws_bytes(q, k_pages, table, max_new=None):
    """Bytes of that workspace."""
    kind = _native.SA_CACHE_BF16 if k_pages.dtype is _torch().bfloat16 else _native.SA_CACHE_E4M3
    _, _, p = _attn_params(q, kind, k_pages.shape, table, max_new, True, 0, None, k_pages.get_device())
    out = ctypes.c_uint64(0)
    with _torch().cuda.device(k_pages.get_device()):
        st = _native.load_library().sparse_attn_paged_ws_bytes(ctypes.byref(p), ctypes.byref(out))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_paged_ws_bytes")
    return int(out.value)


def paged_attn(q, k_pages, v_pages, table, row_start, kv_len, max_new=None, causal=True, window=0, scale=None,
               k_exp=None, v_exp=None, o=None, lse=None, ws=None, stream=None):
    """Attention of the rows of q (bf16 [rows, Hq, 128], any strides that are
    multiples of 8) over their sequences' cached keys: up to the row's own
    token (``causal``), the last ``window`` of these, or all (``causal=False``).
    Query head i reads key head i // (Hq // H).  ``scale`` defaults to
    1 / sqrt(128).  ``max_new`` (default: all rows) bounds the rows of one
    sequence; give it when sequences bring one or a few tokens each.

    Returns (o, lse): bf16 [rows, Hq, 128] and the float32 [rows, Hq] natural
    log-sum-exp of the logits.  A row that sees no key gets zeros and -inf;
    rows of no sequence are left as they were."""
    torch = _torch()
    kind, shape, dev = _cache(k_pages, v_pages, k_exp, v_exp)
    _batch(table, row_start, kv_len, dev)
    n, hq, p = _attn_params(q, kind, shape, table, max_new, causal, window, scale, dev)
    o, fo = _out(o, "o", (n, hq, 128), torch.bfloat16, dev)
    lse, fl = _out(lse, "lse", (n, hq), torch.float32, dev)
    fresh = [t for t, f in ((o, fo), (lse, fl)) if f]
    if ws is None:
        ws = paged_workspace(q, k_pages, table, max_new)
        fresh.append(ws)
    _call("sparse_attn_paged_fwd", dev, stream, fresh, ctypes.byref(p), q.data_ptr(), k_pages.data_ptr(),
          v_pages.data_ptr(), _ptr(k_exp), _ptr(v_exp), table.data_ptr(), row_start.data_ptr(), kv_len.data_ptr(),
          o.data_ptr(), lse.data_ptr(), _scratch(ws, dev), ws.numel())
    return o, lse
