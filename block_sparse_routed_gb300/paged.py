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
  tokens and for single ones;
* ``prefix_attn``: the same where groups of sequences share a prefix.

Nothing here waits for the GPU.  With ``ws`` (a workspace of
``paged_workspace``, or 256 bytes for the two copies)
``sparse_attn_last_device_status(ws)`` tells what the device found wrong.
Without it nobody learns that a sequence was refused (more rows than
``max_new``, a page out of range) or that a call gave up, and outputs that the
call allocated hold in those rows what the memory held before.

``stream``: another stream than the current one waits for nothing by itself;
what the call allocates comes from that stream's memory and may be used on the
current stream once this has waited for the other.
"""

from __future__ import annotations

import ctypes
import functools
import math

from . import _native
from ._native import SA_OK, SaPagedParams, SparseAttnError

PAGE_SIZES = (16, 32, 64, 128)
SCALE = 1.0 / math.sqrt(128.0)


@functools.lru_cache(maxsize=1)
def _env():
    """(torch, bfloat16, float8_e4m3fn, uint8, int32, C library, raw current stream of a device, current device)."""
    import torch

    return (torch, torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int32, _native.load_library(),
            torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)


@functools.lru_cache(maxsize=4096)
def _params(*fields):
    """(C parameters, a reference to them) of a call's sizes: a plain function of numbers."""
    for (name, kind), x in zip(SaPagedParams._fields_[1:], fields):
        bits = 8 * ctypes.sizeof(kind) - 1
        if kind is not ctypes.c_float and not -(1 << bits) <= x < 1 << bits:  # (ctypes would cut it)
            raise ValueError(f"{name}: {x} is out of range")
    p = SaPagedParams(_native.SA_ABI_VERSION, *fields)
    return p, ctypes.byref(p)


def paged_cache(pages, H, page_size=64, dtype="bf16", device="cuda"):
    """An uninitialised cache: (k_pages, v_pages, k_exp, v_exp); the exponents
    are None for ``dtype`` "bf16" and tensors for "e4m3"."""
    import torch

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


def _cache(env, k_pages, v_pages, k_exp, v_exp):
    """Checks the cache's tensors; returns (kind, shape, device index)."""
    shape, dtype, dev = k_pages.shape, k_pages.dtype, k_pages.get_device()
    if dtype is env[1]:
        kind = 0
    elif dtype is env[2]:
        kind = 1
    else:
        raise TypeError("k_pages must be bfloat16 or float8_e4m3fn")
    if dev < 0:
        raise ValueError("k_pages must be a CUDA tensor")
    if v_pages.dtype is not dtype:
        raise TypeError("k_pages and v_pages must have the same dtype")
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must be [pages, H, page_size, 128]")
    if not k_pages.is_contiguous() or not v_pages.is_contiguous() or v_pages.get_device() != dev:
        raise ValueError("k_pages and v_pages must be contiguous and on one device")
    if kind:
        rows = shape[:3]
        for t, name in ((k_exp, "k_exp"), (v_exp, "v_exp")):
            if t is None or t.dtype is not env[3] or t.shape != rows or not t.is_contiguous() or t.get_device() != dev:
                raise ValueError(f"{name}: contiguous uint8 [pages, H, page_size] on the cache's device required")
    elif k_exp is not None or v_exp is not None:
        raise ValueError("a bfloat16 cache has no exponents")
    return kind, shape, dev


def _batch(env, table, row_start, kv_len, dev):
    """Checks the batch; returns (sequences, table width, table stride)."""
    i32 = env[4]
    if table.dtype is not i32 or row_start.dtype is not i32 or kv_len.dtype is not i32:
        raise ValueError("table, row_start and kv_len must be int32")
    if table.get_device() != dev or row_start.get_device() != dev or kv_len.get_device() != dev:
        raise ValueError("table, row_start and kv_len must be on the cache's device")
    if table.dim() != 2:
        raise ValueError("table must be [sequences, width]")
    (n, width), (outer, inner) = table.shape, table.stride()
    if width > 1 and inner != 1:
        raise ValueError("table must have contiguous rows")
    if row_start.dim() != 1 or row_start.numel() != n + 1 or not row_start.is_contiguous():
        raise ValueError("row_start must be contiguous [sequences + 1]")
    if kv_len.dim() != 1 or kv_len.numel() != n or not kv_len.is_contiguous():
        raise ValueError("kv_len must be contiguous [sequences]")
    return n, width, outer


def _rows(env, t, name, dev):
    """Rows [n, heads, 128] (or [1, n, heads, 128]); returns (rows, heads, token stride, head stride)."""
    if t.dtype is not env[1]:
        raise TypeError(f"{name} must be bfloat16")
    shape, stride = t.shape, t.stride()
    if len(shape) == 4 and shape[0] == 1:
        shape, stride = shape[1:], stride[1:]
    if len(shape) != 3 or shape[2] != 128:
        raise ValueError(f"{name} must be [rows, heads, 128], got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the cache's device")
    n, h, _ = shape
    ts, hs, ds = stride
    # strides of dimensions of one element mean nothing
    ts, hs = (ts if n > 1 else 0), (hs if h > 1 else 0)
    if ds != 1 or ts % 8 or hs % 8:
        raise ValueError(f"{name}: contiguous last dimension and strides that are multiples of 8 required")
    return n, h, ts, hs


def _given(t, name, shape, dtype, dev):
    """Checks an output of the given shape (a leading 1 is allowed, as in the rows)."""
    if (t.dtype is not dtype or (t.shape != shape and t.shape != (1, *shape)) or not t.is_contiguous()
            or t.get_device() != dev):
        raise ValueError(f"{name}: contiguous {dtype} {list(shape)} on the cache's device required")
    return t


def _scratch(env, ws, dev, least):
    if ws.dtype is not env[3] or not ws.is_contiguous() or ws.get_device() != dev or ws.numel() < least:
        raise ValueError(f"ws must be a contiguous uint8 tensor of {least} bytes at least, on the cache's device")
    return ws.data_ptr()


def _new(env, stream, like, shape, dtype):
    """A tensor that a call on ``stream`` fills.  On another stream than the
    current one it comes from that stream's pool (what the current stream has
    freed may still be in use there), and is kept for the current one, where
    the caller may use it."""
    if stream is None or stream.cuda_stream == env[6](like.get_device()):
        return env[0].empty(shape, dtype=dtype, device=like.device)
    here = env[0].cuda.current_stream(like.device)
    with env[0].cuda.stream(stream):
        t = env[0].empty(shape, dtype=dtype, device=like.device)
    t.record_stream(here)
    return t


def _call(env, name, dev, stream, args):
    """Runs a C entry point on ``stream`` (default: the device's current one)."""
    raw = env[6](dev) if stream is None else stream.cuda_stream
    fn = getattr(env[5], name)
    if env[7]() == dev:
        st = fn(*args, raw or None)
    else:
        with env[0].cuda.device(dev):
            st = fn(*args, raw or None)
    if st != SA_OK:
        raise SparseAttnError(st, name)


def cache_write(k, v, k_pages, v_pages, table, row_start, kv_len, k_exp=None, v_exp=None, ws=None, stream=None):
    """Writes the rows of k and v (bf16 [rows, H, 128], any strides that are
    multiples of 8) to their sequences' pages, quantised for an E4M3 cache."""
    env = _env()
    kind, (pages, H, ps, d), dev = _cache(env, k_pages, v_pages, k_exp, v_exp)
    seqs, width, outer = _batch(env, table, row_start, kv_len, dev)
    n, h, kt, kh = _rows(env, k, "k", dev)
    nv, hv, vt, vh = _rows(env, v, "v", dev)
    if n != nv or h != H or hv != H:
        raise ValueError("k and v must both be [rows, H, 128] with the cache's H")
    _, p = _params(kind, pages, H, ps, d, seqs, width, outer, n, n, H, 1, 0, 1.0, kt, kh, vt, vh)
    _call(env, "sparse_attn_cache_write", dev, stream, (
        p, k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_exp.data_ptr() if kind else None,
        v_exp.data_ptr() if kind else None, table.data_ptr(), row_start.data_ptr(), kv_len.data_ptr(),
        None if ws is None else _scratch(env, ws, dev, 256)))


def cache_read(k_pages, v_pages, table, row_start, kv_len, rows=None, k_exp=None, v_exp=None, k=None, v=None, ws=None,
               stream=None):
    """The rows of every sequence as bf16 (k, v) [rows, H, 128].  ``rows`` (the
    last row_start) sizes the outputs when k and v are not given."""
    env = _env()
    kind, (pages, H, ps, d), dev = _cache(env, k_pages, v_pages, k_exp, v_exp)
    seqs, width, outer = _batch(env, table, row_start, kv_len, dev)
    if rows is None:
        if k is None:
            raise ValueError("give rows, or k and v")
        rows = _rows(env, k, "k", dev)[0]
    k, v = (_new(env, stream, k_pages, (rows, H, 128), env[1]) if t is None
            else _given(t, name, (rows, H, 128), env[1], dev) for t, name in ((k, "k"), (v, "v")))
    _, p = _params(kind, pages, H, ps, d, seqs, width, outer, rows, rows, H, 1, 0, 1.0, 0, 0, 0, 0)
    _call(env, "sparse_attn_cache_read", dev, stream, (
        p, k_pages.data_ptr(), v_pages.data_ptr(), k_exp.data_ptr() if kind else None,
        v_exp.data_ptr() if kind else None, table.data_ptr(), row_start.data_ptr(), kv_len.data_ptr(), k.data_ptr(),
        v.data_ptr(), None if ws is None else _scratch(env, ws, dev, 256)))
    return k, v


@functools.lru_cache(maxsize=4096)
def _ws_bytes(*fields):
    """Bytes of a call's workspace: a plain function of numbers."""
    out = ctypes.c_uint64(0)
    st = _native.load_library().sparse_attn_paged_ws_bytes(_params(*fields)[1], ctypes.byref(out))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_paged_ws_bytes")
    return int(out.value)


def paged_ws_bytes(q, k_pages, table, max_new=None):
    """Bytes of the workspace of ``paged_attn`` calls of these sizes."""
    env = _env()
    n, hq, _, _ = _rows(env, q, "q", q.get_device())
    pages, H, ps, d = k_pages.shape
    if hq < 1 or H < 1 or hq % H:
        raise ValueError("q's heads must be a multiple of the cache's")
    max_new = n if max_new is None else min(int(max_new), n)
    return _ws_bytes(1 if k_pages.dtype is env[2] else 0, pages, H, ps, d, table.shape[0], table.shape[1], 0, n,
                     max_new, hq, 1, 0, 1.0, 0, 0, 0, 0)


def paged_workspace(q, k_pages, table, max_new=None):
    """A workspace for ``paged_attn`` calls of these sizes.  It belongs to one
    stream at a time; two captured graphs that may run at once need two."""
    return _env()[0].empty(paged_ws_bytes(q, k_pages, table, max_new), dtype=_env()[3], device=k_pages.device)


def paged_attn(q, k_pages, v_pages, table, row_start, kv_len, max_new=None, causal=True, window=0, scale=None,
               k_exp=None, v_exp=None, o=None, lse=None, ws=None, stream=None):
    """Attention of the rows of q (bf16 [rows, Hq, 128], any strides that are
    multiples of 8) over their sequences' cached keys: up to the row's own
    token (``causal``), the last ``window`` of these, or all (``causal=False``).
    Query head i reads key head i // (Hq // H).  ``scale`` (> 0) defaults to
    1 / sqrt(128).  ``max_new`` (default: all rows) bounds the rows of one
    sequence; give it when sequences bring one or a few tokens each.

    Returns (o, lse): bf16 [rows, Hq, 128] and the float32 [rows, Hq] natural
    log-sum-exp of the logits.  A row that sees no key gets zeros and -inf;
    rows of no sequence are left as they were."""
    env = _env()
    kind, (pages, H, ps, d), dev = _cache(env, k_pages, v_pages, k_exp, v_exp)
    seqs, width, outer = _batch(env, table, row_start, kv_len, dev)
    n, hq, qt, qh = _rows(env, q, "q", dev)
    if hq < 1 or H < 1 or hq % H:
        raise ValueError("q's heads must be a multiple of the cache's")
    if window < 0 or (window and not causal):
        raise ValueError("window: 0, or a positive number with causal=True")
    if window > 0x7FFFFFFF:  # more tokens than a sequence can have
        window = 0x7FFFFFFF
    max_new = n if max_new is None or max_new > n else max_new
    if max_new < 0:
        raise ValueError("max_new must not be negative")
    if o is None:
        o = _new(env, stream, k_pages, (n, hq, 128), env[1])
    else:
        _given(o, "o", (n, hq, 128), env[1], dev)
    if lse is None:
        lse = _new(env, stream, k_pages, (n, hq), env[0].float32)
    else:
        _given(lse, "lse", (n, hq), env[0].float32, dev)
    fields = (kind, pages, H, ps, d, seqs, width, outer, n, max_new, hq, 1 if causal else 0, window,
              SCALE if scale is None else scale, qt, qh, 0, 0)
    if ws is None:
        ws = _new(env, stream, k_pages, (_ws_bytes(*fields),), env[3])
    _, p = _params(*fields)
    _call(env, "sparse_attn_paged_fwd", dev, stream, (
        p, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_exp.data_ptr() if kind else None,
        v_exp.data_ptr() if kind else None, table.data_ptr(), row_start.data_ptr(), kv_len.data_ptr(), o.data_ptr(),
        lse.data_ptr(), _scratch(env, ws, dev, 0), ws.numel()))
    return o, lse


def _groups(env, group_start, prefix_len, dev):
    """Checks the groups; returns their number."""
    for t, name in ((group_start, "group_start"), (prefix_len, "prefix_len")):
        if t.dtype is not env[4] or t.dim() != 1 or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"{name}: contiguous int32 vector on the cache's device required")
    if group_start.numel() != prefix_len.numel() + 1:
        raise ValueError("group_start must be [groups + 1] and prefix_len [groups]")
    return prefix_len.numel()


@functools.lru_cache(maxsize=4096)
def _prefix_ws_bytes(groups, *fields):
    """Bytes of a call's workspace: a plain function of numbers."""
    out = ctypes.c_uint64(0)
    st = _native.load_library().sparse_attn_prefix_ws_bytes(_params(*fields)[1], groups, ctypes.byref(out))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_prefix_ws_bytes")
    return int(out.value)


def prefix_ws_bytes(q, k_pages, table, group_start, max_new=None):
    """Bytes of the workspace of ``prefix_attn`` calls of these sizes."""
    env = _env()
    n, hq, _, _ = _rows(env, q, "q", q.get_device())
    pages, H, ps, d = k_pages.shape
    if hq < 1 or H < 1 or hq % H:
        raise ValueError("q's heads must be a multiple of the cache's")
    max_new = n if max_new is None else min(int(max_new), n)
    return _prefix_ws_bytes(group_start.numel() - 1, 1 if k_pages.dtype is env[2] else 0, pages, H, ps, d, table.shape[0],
                            table.shape[1], 0, n, max_new, hq, 1, 0, 1.0, 0, 0, 0, 0)


def prefix_workspace(q, k_pages, table, group_start, max_new=None):
    """A workspace for ``prefix_attn`` calls of these sizes, as ``paged_workspace``."""
    return _env()[0].empty(prefix_ws_bytes(q, k_pages, table, group_start, max_new), dtype=_env()[3], device=k_pages.device)


def prefix_attn(q, k_pages, v_pages, table, row_start, kv_len, group_start, prefix_len, max_new=None, causal=True,
                scale=None, k_exp=None, v_exp=None, o=None, lse=None, ws=None, stream=None):
    """``paged_attn`` for a batch in which groups of sequences begin with the
    same tokens, whose keys are read once for all rows of the group.

    ``group_start`` (int32 [groups + 1], ascending) and ``prefix_len`` (int32
    [groups]), on the GPU: the sequences group_start[g] .. group_start[g + 1] - 1
    begin with the same prefix_len[g] tokens.  Those in whole pages are read
    once, from the pages of the group's first sequence that has rows, which the
    others' rows of ``table`` name too; all others by each sequence's own row.  A
    sequence's rows must lie behind the shared pages; of one without rows (an
    empty slot) nothing has to agree with its group.  There is no window.  A
    batch of one sequence, or without rows, shares nothing: its groups are not
    looked at.

    Returns (o, lse) as ``paged_attn``, equal up to the order of sums.  It pays
    where the shared keys, counted once for each sequence, are about 130000 or
    more; below, ``paged_attn`` takes less time."""
    env = _env()
    kind, (pages, H, ps, d), dev = _cache(env, k_pages, v_pages, k_exp, v_exp)
    seqs, width, outer = _batch(env, table, row_start, kv_len, dev)
    groups = _groups(env, group_start, prefix_len, dev)
    n, hq, qt, qh = _rows(env, q, "q", dev)
    if hq < 1 or H < 1 or hq % H:
        raise ValueError("q's heads must be a multiple of the cache's")
    max_new = n if max_new is None or max_new > n else max_new
    if max_new < 0:
        raise ValueError("max_new must not be negative")
    if o is None:
        o = _new(env, stream, k_pages, (n, hq, 128), env[1])
    else:
        _given(o, "o", (n, hq, 128), env[1], dev)
    if lse is None:
        lse = _new(env, stream, k_pages, (n, hq), env[0].float32)
    else:
        _given(lse, "lse", (n, hq), env[0].float32, dev)
    fields = (kind, pages, H, ps, d, seqs, width, outer, n, max_new, hq, 1 if causal else 0, 0,
              SCALE if scale is None else scale, qt, qh, 0, 0)
    if ws is None:
        ws = _new(env, stream, k_pages, (_prefix_ws_bytes(groups, *fields),), env[3])
    _, p = _params(*fields)
    _call(env, "sparse_attn_prefix_fwd", dev, stream, (
        p, groups, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_exp.data_ptr() if kind else None,
        v_exp.data_ptr() if kind else None, table.data_ptr(), row_start.data_ptr(), kv_len.data_ptr(),
        group_start.data_ptr(), prefix_len.data_ptr(), o.data_ptr(), lse.data_ptr(), _scratch(env, ws, dev, 0), ws.numel()))
    return o, lse
