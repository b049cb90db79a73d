"""Shared prefixes, weights of cached keys and eviction without a GPU: pins of the
oracle, the C structures, and every refusal that the host makes before anything
is enqueued."""

import ctypes
import math

import numpy as np
import pytest

from oracle import paged as OP

from .test_paged_host import A, BIG, _p, native  # noqa: F401


# ---- the oracle

def test_a_row_gives_one_for_each_head_of_the_group():
    rng = np.random.default_rng(0)
    k, v, q = rng.standard_normal((9, 2, 128)), rng.standard_normal((9, 2, 128)), rng.standard_normal((3, 6, 128))
    pos = [6, 7, 8]
    _, lse, _, _ = OP.paged_attention(q, k, v, pos, 9)
    w, slack, count = OP.received(q, lse, k, pos, 9)
    assert np.allclose(w.sum(1), 9) and count[:, 0].tolist() == [9, 9] and count[:, 8].tolist() == [3, 3]
    assert np.all(w[:, 8] < 3) and np.all(slack >= 0)
    # by hand: the last key, seen by the last row alone
    for h in range(2):
        x = q[2, 3 * h:3 * h + 3] @ k[8, h] / math.sqrt(128)
        assert np.isclose(w[h, 8], np.exp(x - lse[2, 3 * h:3 * h + 3]).sum())
    w2, _, c2 = OP.received(q, lse, k, pos, 9, window=2)
    assert np.all(c2[:, :5] == 0) and np.all(w2[:, :5] == 0) and c2[0].tolist() == [0] * 5 + [3, 6, 6, 3]
    lse[1] = -np.inf
    assert np.all(OP.received(q, lse, k, pos, 9)[2][:, 0] == 6)


def test_survivors_by_hand():
    w = np.array([0.0, 5.0, 1.0, 3.0, 3.0, 0.5, 9.0])
    assert OP.survivors(w, 7, 0, 0) == list(range(7))
    assert OP.survivors(w, 3, 0, 0) == [1, 3, 6]           # of the equal ones the earlier
    assert OP.survivors(w, 4, 0, 0) == [1, 3, 4, 6]
    assert OP.survivors(w, 3, 1, 1) == [0, 1, 6]
    assert OP.survivors(w, 3, 1, 2) == [0, 5, 6]           # nothing to choose
    w = np.array([-0.0, 0.0, math.nan, math.inf, -1.0])
    assert OP.survivors(w, 1, 0, 0) == [2] and OP.survivors(w, 3, 0, 0) == [0, 2, 3]


# ---- the C entry points

E_FIELDS = dict(keep=64, first=4, last=8, to_width=4, to_stride=4)


def _evict(native, p, kp=A, vp=A, ke=A, ve=A, w=A, table=A, kl=A, to=A, kept=A, new=2 * A, ws=A, e=E_FIELDS):
    ep = None if e is None else native.SaEvictParams(*e.values())
    return native.load_library().sparse_attn_cache_evict(ctypes.byref(p), None if ep is None else ctypes.byref(ep), kp, vp, ke, ve, w,
                                                         table, kl, to, kept, new, ws, None)


def _weigh(native, p, first=0, acc=1, q=A, lse=A, kp=A, ke=A, table=A, rs=A, kl=A, w=A, ws=A, n=BIG):
    return native.load_library().sparse_attn_cache_weigh(ctypes.byref(p), first, acc, q, lse, kp, ke, table, rs, kl, w, ws, n, None)


def _prefix(native, p, groups=2, q=A, kp=A, vp=A, ke=A, ve=A, table=A, rs=A, kl=A, gs=A, pl=A, o=A, lse=A, ws=A, n=BIG):
    return native.load_library().sparse_attn_prefix_fwd(ctypes.byref(p), groups, q, kp, vp, ke, ve, table, rs, kl, gs, pl, o, lse, ws, n,
                                                        None)


CALLS = (_evict, _weigh, _prefix)


def test_struct_size(native):  # noqa: F811
    assert ctypes.sizeof(native.SaEvictParams) == 24


@pytest.mark.parametrize("bad", [dict(ver=2), dict(kind=2), dict(pages=0), dict(H=0), dict(page_size=48), dict(seqs=-1),
                                 dict(rows=-1), dict(max_new=-1), dict(table_width=-1), dict(table_stride=-4)])
def test_every_call_refuses_bad_fields(native, bad):  # noqa: F811
    for call in CALLS:
        assert call(native, _p(native, **bad)) == native.SA_EINVAL


@pytest.mark.parametrize("bad", [dict(D=64), dict(pages=1 << 25), dict(pages=(1 << 31) - 1, H=2), dict(table_width=1 << 25)])
def test_every_call_refuses_unsupported_sizes(native, bad):  # noqa: F811
    for call in CALLS:
        assert call(native, _p(native, **bad)) == native.SA_EUNSUPPORTED


@pytest.mark.parametrize("bad", [dict(kp=None), dict(kl=None), dict(table=None), dict(kp=A + 8), dict(table=A + 2), dict(kl=A + 2),
                                 dict(ws=A + 128)])
def test_every_call_refuses_bad_pointers(native, bad):  # noqa: F811
    for call in CALLS:
        assert call(native, _p(native), **bad) == native.SA_EINVAL


@pytest.mark.parametrize("bad", [dict(ke=None), dict(ke=A + 8)])
def test_every_call_refuses_bad_exponents(native, bad):  # noqa: F811
    for call in CALLS:
        assert call(native, _p(native, kind=1), **bad) == native.SA_EINVAL


@pytest.mark.parametrize("bad", [dict(first=-1), dict(acc=2), dict(acc=-1), dict(q=None), dict(lse=None), dict(w=None), dict(ws=None),
                                 dict(q=A + 2), dict(lse=A + 2), dict(w=A + 4), dict(rs=None), dict(n=255)])
def test_weigh_refuses(native, bad):  # noqa: F811
    assert _weigh(native, _p(native), **bad) == native.SA_EINVAL


@pytest.mark.parametrize("bad", [dict(Hq=3), dict(Hq=0), dict(causal=2), dict(window=-1), dict(window=3, causal=0), dict(scale=0.0),
                                 dict(scale=math.inf), dict(scale=math.nan), dict(at=-8), dict(ah=4)])
def test_weigh_and_prefix_refuse_bad_attention(native, bad):  # noqa: F811
    assert _weigh(native, _p(native, **bad)) == native.SA_EINVAL
    assert _prefix(native, _p(native, **bad)) == native.SA_EINVAL


def test_weigh_refuses_scales_past_its_range(native):  # noqa: F811
    for scale in (2.0 ** -101, 2.0 ** 101):
        assert _weigh(native, _p(native, scale=scale)) == native.SA_EUNSUPPORTED


@pytest.mark.parametrize("bad", [dict(groups=-1), dict(gs=None), dict(pl=None), dict(gs=A + 2), dict(pl=A + 1), dict(q=None),
                                 dict(o=None), dict(o=A + 16), dict(lse=A + 2), dict(ws=None), dict(vp=None), dict(rs=None), dict(n=255)])
def test_prefix_refuses(native, bad):  # noqa: F811
    assert _prefix(native, _p(native), **bad) == native.SA_EINVAL


def test_prefix_has_no_window(native):  # noqa: F811
    p, out = _p(native, window=5), ctypes.c_uint64()
    assert _prefix(native, p) == native.SA_EINVAL
    assert native.load_library().sparse_attn_prefix_ws_bytes(ctypes.byref(p), 2, ctypes.byref(out)) == native.SA_EINVAL
    p = _p(native)
    assert native.load_library().sparse_attn_prefix_ws_bytes(ctypes.byref(p), 2, None) == native.SA_EINVAL
    assert native.load_library().sparse_attn_prefix_ws_bytes(ctypes.byref(p), 2, ctypes.byref(out)) == native.SA_OK and out.value > 7 * 4 * 1056
    assert native.load_library().sparse_attn_weigh_ws_bytes(ctypes.byref(p), None) == native.SA_EINVAL


@pytest.mark.parametrize("bad", [dict(keep=0), dict(keep=-5), dict(first=-1), dict(last=-1), dict(first=60, last=5), dict(to_width=-1),
                                 dict(to_stride=-1), dict(first=(1 << 31) - 1, last=(1 << 31) - 1)])
def test_evict_refuses_bad_numbers(native, bad):  # noqa: F811
    assert _evict(native, _p(native), e=dict(E_FIELDS, **bad)) == native.SA_EINVAL


@pytest.mark.parametrize("bad", [dict(e=None), dict(w=None), dict(kept=None), dict(new=None), dict(w=A + 4), dict(to=A + 2), dict(kept=A + 2),
                                 dict(new=A + 1), dict(new=A), dict(vp=None)])
def test_evict_refuses(native, bad):  # noqa: F811
    assert _evict(native, _p(native), **bad) == native.SA_EINVAL


@pytest.mark.parametrize("kw", [dict(seqs=1 << 26), dict(table_width=(1 << 24) + 1)])
def test_evict_refuses_unsupported_sizes(native, kw):  # noqa: F811
    assert _evict(native, _p(native, **kw)) == native.SA_EUNSUPPORTED
    assert _evict(native, _p(native), e=dict(E_FIELDS, keep=(1 << 30) + 1)) == native.SA_EUNSUPPORTED


def test_python_refuses_without_a_gpu():
    """What the Python layer checks before it looks for a device."""
    torch = pytest.importorskip("torch")
    import block_sparse_routed_gb300 as bsr

    k = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    w = bsr.cache_weights(k)
    assert w.shape == (4, 2, 16) and w.dtype == torch.float32 and not w.any()
    i32 = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        bsr.cache_evict(k, k, w, i32[None], i32, 5)
    with pytest.raises(ValueError):
        bsr.cache_weigh(k[0, :, :, :], torch.zeros(2, 16), w, k, i32[None], i32, i32)
    with pytest.raises(ValueError):
        bsr.prefix_attn(k[0], k, k, i32[None], torch.zeros(2, dtype=torch.int32), i32, i32, i32[:0])
