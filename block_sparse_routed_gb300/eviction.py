"""Eviction from a paged cache by the attention weight that its keys received.

``weights`` (float32 [pages, H, page_size]) lies beside the pages of ``paged.py``
and belongs to the token in a page's slot.

* ``cache_weigh``: adds what the rows of a call give to the keys that they
  see, from their ``lse``;
* ``cache_evict``: every sequence and key head keeps its first and last tokens
  and the most weighted of the others, moved together.

A decoding loop calls ``cache_write``, ``paged_attn`` (or ``prefix_attn``) and
``cache_weigh`` in each step, and ``cache_evict`` when a sequence is over its
budget.  After a long prompt, ``accumulate=False`` with its last rows alone
weighs the prompt by what they attend to.

Nothing here waits for the GPU; ``ws``, ``stream`` and the status are as in
``paged.py``.
"""

from __future__ import annotations

import ctypes
import functools

from . import _native
from ._native import SA_OK, SaEvictParams, SparseAttnError
from .paged import SCALE, _batch, _cache, _call, _env, _given, _new, _params, _rows, _scratch

_INT32 = 0x7FFFFFFF
_STATUS_BYTES = 256  # of a workspace, at its start


def cache_weights(k_pages):
    """Weights for a cache: zeros, float32 [pages, H, page_size]."""
    import torch

    return torch.zeros(k_pages.shape[:3], dtype=torch.float32, device=k_pages.device)


def _weights(env, weights, shape, dev):
    if (weights.dtype is not env[0].float32 or weights.shape != shape or not weights.is_contiguous()
            or weights.get_device() != dev):
        raise ValueError("weights: contiguous float32 [pages, H, page_size] on the cache's device required")
    return weights.data_ptr()


@functools.lru_cache(maxsize=4096)
def _weigh_ws_bytes(*fields):
    """Bytes of a call's workspace: a plain function of numbers."""
    out = ctypes.c_uint64(0)
    st = _native.load_library().sparse_attn_weigh_ws_bytes(_params(*fields)[1], ctypes.byref(out))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_weigh_ws_bytes")
    return int(out.value)


def weigh_workspace(q, k_pages, table, max_new=None):
    """A workspace for ``cache_weigh`` calls of these sizes, as ``paged_workspace``."""
    env = _env()
    n, hq, _, _ = _rows(env, q, "q", q.get_device())
    pages, H, ps, d = k_pages.shape
    if hq < 1 or H < 1 or hq % H:
        raise ValueError("q's heads must be a multiple of the cache's")
    max_new = n if max_new is None else min(int(max_new), n)
    size = _weigh_ws_bytes(1 if k_pages.dtype is env[2] else 0, pages, H, ps, d, table.shape[0], table.shape[1], 0, n, max_new,
                           hq, 1, 0, 1.0, 0, 0, 0, 0)
    return env[0].empty(size, dtype=env[3], device=k_pages.device)


def cache_weigh(q, lse, weights, k_pages, table, row_start, kv_len, max_new=None, causal=True, window=0, scale=None,
                first=0, accumulate=True, k_exp=None, ws=None, stream=None):
    """Adds to the weight of each cached key at position ``first`` or later the
    sum of exp(logit - lse) over the rows of q that see it and the query heads
    that read its head.  ``q``, ``lse``, ``max_new``, ``causal``, ``window`` and
    ``scale`` are those of the ``paged_attn`` or ``prefix_attn`` call that gave
    ``lse``.  The call's own tokens, and with ``accumulate=False`` all tokens of
    the sequences that have rows, start from 0.  Returns ``weights``."""
    env = _env()
    kind, (pages, H, ps, d), dev = _cache(env, k_pages, k_pages, k_exp, k_exp)
    seqs, width, outer = _batch(env, table, row_start, kv_len, dev)
    n, hq, qt, qh = _rows(env, q, "q", dev)
    if hq < 1 or H < 1 or hq % H:
        raise ValueError("q's heads must be a multiple of the cache's")
    if window < 0 or (window and not causal):
        raise ValueError("window: 0, or a positive number with causal=True")
    if first < 0:
        raise ValueError("first must not be negative")
    max_new = n if max_new is None or max_new > n else max_new
    if max_new < 0:
        raise ValueError("max_new must not be negative")
    _given(lse, "lse", (n, hq), env[0].float32, dev)
    w = _weights(env, weights, (pages, H, ps), dev)
    fields = (kind, pages, H, ps, d, seqs, width, outer, n, max_new, hq, 1 if causal else 0, min(window, _INT32),
              SCALE if scale is None else scale, qt, qh, 0, 0)
    at = size = 0
    if ws is None:
        need = _weigh_ws_bytes(*fields)
        if need > _STATUS_BYTES:
            ws = _new(env, stream, k_pages, (need,), env[3])
    if ws is not None:
        at, size = _scratch(env, ws, dev, _STATUS_BYTES), ws.numel()
    _, p = _params(*fields)
    _call(env, "sparse_attn_cache_weigh", dev, stream, (
        p, min(first, _INT32), 1 if accumulate else 0, q.data_ptr(), lse.data_ptr(), k_pages.data_ptr(),
        k_exp.data_ptr() if kind else None, table.data_ptr(), row_start.data_ptr(), kv_len.data_ptr(), w,
        at or None, size))
    return weights


@functools.lru_cache(maxsize=4096)
def _evict_params(*fields):
    e = SaEvictParams(*fields)
    return e, ctypes.byref(e)


def cache_evict(k_pages, v_pages, weights, table, kv_len, keep, first=0, last=0, to_table=None, k_exp=None, v_exp=None,
                kept=None, new_len=None, ws=None, stream=None):
    """Each key head of a sequence with more than ``keep`` tokens keeps its
    ``first`` and ``last`` ones and, up to ``keep``, those of the others with the
    largest weights (of equal ones the earlier).  K, V, exponents and weights
    of what stays move in order to the positions 0 .., in place or to the pages
    of ``to_table`` (int32 [sequences, width], pages that hold none of these
    sequences' tokens).

    Returns (kept, new_len): int32 [sequences, H, keep], the former position of
    each token that stayed (-1 past the new length), and int32 [sequences], the
    new ``kv_len``.  In place, pages past a sequence's new length are free, and
    pages that several sequences share must lie below ``first``."""
    env = _env()
    kind, (pages, H, ps, d), dev = _cache(env, k_pages, v_pages, k_exp, v_exp)
    i32 = env[4]
    if table.dtype is not i32 or kv_len.dtype is not i32 or table.get_device() != dev or kv_len.get_device() != dev:
        raise ValueError("table and kv_len must be int32 and on the cache's device")
    tables = []
    for t, name in ((table, "table"), (to_table, "to_table")):
        if t is None:
            tables.append((0, 0))
            continue
        if t.dtype is not i32 or t.get_device() != dev:
            raise ValueError(f"{name} must be int32 and on the cache's device")
        if t.dim() != 2 or t.shape[0] != table.shape[0]:
            raise ValueError(f"{name} must be [sequences, width]")
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have contiguous rows")
        tables.append((t.shape[1], t.stride(0)))
    if to_table is not None and to_table.numel() == 0 and table.shape[0]:
        raise ValueError("to_table has no pages")
    (width, outer), (to_width, to_outer) = tables
    seqs = table.shape[0]
    if kv_len.dim() != 1 or kv_len.numel() != seqs or not kv_len.is_contiguous():
        raise ValueError("kv_len must be contiguous [sequences]")
    if keep < 1 or keep > _INT32:
        raise ValueError("keep must be at least 1 (and below 2^31)")
    if first < 0 or last < 0 or first + last > keep:
        raise ValueError("first and last must not be negative, nor together more than keep")
    w = _weights(env, weights, (pages, H, ps), dev)
    if kept is None:
        kept = _new(env, stream, k_pages, (seqs, H, keep), i32)
    else:
        _given(kept, "kept", (seqs, H, keep), i32, dev)
    if new_len is None:
        new_len = _new(env, stream, k_pages, (seqs,), i32)
    else:
        _given(new_len, "new_len", (seqs,), i32, dev)
    _, p = _params(kind, pages, H, ps, d, seqs, width, outer, 0, 0, H, 1, 0, 1.0, 0, 0, 0, 0)
    _, e = _evict_params(keep, first, last, to_width, to_outer)
    _call(env, "sparse_attn_cache_evict", dev, stream, (
        p, e, k_pages.data_ptr(), v_pages.data_ptr(), k_exp.data_ptr() if kind else None,
        v_exp.data_ptr() if kind else None, w, table.data_ptr(), kv_len.data_ptr(),
        None if to_table is None else to_table.data_ptr(), kept.data_ptr(), new_len.data_ptr(),
        None if ws is None else _scratch(env, ws, dev, 256)))
    return kept, new_len
