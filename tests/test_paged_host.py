"""The paged cache without a GPU: the oracle's own pins, the C structure, and
every refusal that the host makes before anything is enqueued."""

import ctypes

import numpy as np
import pytest

import oracle as O
from oracle import paged as OP


@pytest.fixture(scope="module")
def native():
    import os

    from block_sparse_routed_gb300 import _native
    from block_sparse_routed_gb300.build import LIB_PATH, build

    if not os.path.exists(LIB_PATH):
        build()
    _native.load_library()
    return _native


# ---- the oracle

def test_e4m3_values_are_the_formats():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(OP.e4m3_values(), want, equal_nan=True)


def test_quantised_rows_match_an_independent_rounding():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    for scale in (1.0, 1e-3, 3e20, 1e-36, 448.0, 0.0):
        x = torch.from_numpy((rng.standard_normal(128) * scale).astype(np.float32)).bfloat16()
        bits = x.view(torch.int16).numpy().view(np.uint16)
        codes, byte = OP.quantise_row(bits)
        e = byte - 127
        amax = x.double().abs().max().item()
        assert amax <= 448 * 2.0 ** e and (e == -126 or amax > 448 * 2.0 ** (e - 1))
        want = (x.double() * 2.0 ** -e).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes, want)
        # half a step of the format, or half of its smallest one
        back = OP.dequantise(codes[None], np.array([byte]))[0]
        ref = O.decode_bf16(bits)
        assert np.all(np.abs(back - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * 2.0 ** e))


def test_attention_of_the_last_row_is_softmax_over_all():
    rng = np.random.default_rng(0)
    k, v, q = rng.standard_normal((9, 2, 128)), rng.standard_normal((9, 2, 128)), rng.standard_normal((1, 4, 128))
    o, lse, _, _ = OP.paged_attention(q, k, v, [8], 9)
    for h in range(4):
        x = k[:, h // 2] @ q[0, h] / np.sqrt(128)
        w = np.exp(x) / np.exp(x).sum()
        assert np.allclose(o[0, h], w @ v[:, h // 2]) and np.isclose(lse[0, h], np.log(np.exp(x).sum()))
    assert OP.visible(8, 9, True, 0) == (0, 9) and OP.visible(3, 9, True, 2) == (2, 4)
    assert OP.visible(-2, 9, True, 0) == (0, 0) and OP.visible(-2, 9, False, 0) == (0, 9)
    o, lse, _, _ = OP.paged_attention(q, k, v, [-1], 9)
    assert not o.any() and np.all(lse == -np.inf)


# ---- the C entry points

FIELDS = dict(kind=0, pages=10, H=2, page_size=64, D=128, seqs=3, table_width=4, table_stride=4, rows=7, max_new=7,
              Hq=4, causal=1, window=0, scale=0.1, at=512, ah=128, bt=512, bh=128)


def _p(native, ver=None, **kw):
    f = dict(FIELDS, **kw)
    return native.SaPagedParams(native.SA_ABI_VERSION if ver is None else ver, *f.values())


A = 1 << 20  # an aligned address that no path here may touch
BIG = 1 << 40


def _write(native, p, k=A, v=A, kp=A, vp=A, ke=A, ve=A, table=A, rs=A, kl=A, ws=A):
    return native.load_library().sparse_attn_cache_write(ctypes.byref(p), k, v, kp, vp, ke, ve, table, rs, kl, ws, None)


def _read(native, p, k=A, v=A, kp=A, vp=A, ke=A, ve=A, table=A, rs=A, kl=A, ws=A):
    return native.load_library().sparse_attn_cache_read(ctypes.byref(p), kp, vp, ke, ve, table, rs, kl, k, v, ws, None)


def _fwd(native, p, q=A, kp=A, vp=A, ke=A, ve=A, table=A, rs=A, kl=A, o=A, lse=A, ws=A, n=BIG):
    return native.load_library().sparse_attn_paged_fwd(ctypes.byref(p), q, kp, vp, ke, ve, table, rs, kl, o, lse, ws, n,
                                                       None)


def test_struct_size(native):
    assert ctypes.sizeof(native.SaPagedParams) == 96


@pytest.mark.parametrize("bad", [dict(ver=2), dict(kind=2), dict(pages=0), dict(H=0), dict(page_size=48),
                                 dict(page_size=256), dict(seqs=-1), dict(rows=-1), dict(max_new=-1),
                                 dict(table_width=-1), dict(table_stride=-4)])
def test_every_call_refuses_bad_fields(native, bad):
    p = _p(native, **bad)
    for call in (_write, _read, _fwd):
        assert call(native, p) == native.SA_EINVAL
    assert native.load_library().sparse_attn_paged_ws_bytes(ctypes.byref(p), ctypes.byref(ctypes.c_uint64())) == \
        native.SA_EINVAL


@pytest.mark.parametrize("bad", [dict(D=64), dict(pages=1 << 25), dict(pages=(1 << 31) - 1, H=2),
                                 dict(table_width=1 << 25), dict(rows=(1 << 30), H=2, Hq=2)])
def test_every_call_refuses_unsupported_sizes(native, bad):
    p = _p(native, **bad)
    for call in (_write, _read, _fwd):
        assert call(native, p) == native.SA_EUNSUPPORTED


@pytest.mark.parametrize("bad", [dict(kp=None), dict(vp=None), dict(rs=None), dict(kl=None), dict(table=None),
                                 dict(kp=A + 8), dict(vp=A + 2), dict(table=A + 2), dict(rs=A + 1), dict(kl=A + 2),
                                 dict(ws=A + 128)])
def test_every_call_refuses_bad_pointers(native, bad):
    for kind in (0, 1):
        p = _p(native, kind=kind)
        for call in (_write, _read, _fwd):
            assert call(native, p, **bad) == native.SA_EINVAL
    p = _p(native, kind=1)
    for call in (_write, _read, _fwd):
        assert call(native, p, ke=None) == native.SA_EINVAL
        assert call(native, p, ve=A + 4) == native.SA_EINVAL


def test_copies_refuse_their_own(native):
    p = _p(native)
    for bad in (dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 2)):
        assert _write(native, p, **bad) == native.SA_EINVAL
        assert _read(native, p, **bad) == native.SA_EINVAL
    for f in ("at", "ah", "bt", "bh"):
        for x in (-8, 4):
            assert _write(native, _p(native, **{f: x})) == native.SA_EINVAL


def test_attention_refuses_its_own(native):
    E = native.SA_EINVAL
    for bad in (dict(Hq=3), dict(Hq=0), dict(causal=2), dict(window=-1), dict(causal=0, window=4),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=0.0), dict(scale=-1.0), dict(at=4), dict(ah=-128)):
        assert _fwd(native, _p(native, **bad)) == E, bad
    p = _p(native)
    for bad in (dict(q=None), dict(o=None), dict(ws=None), dict(q=A + 8), dict(o=A + 16), dict(lse=A + 2), dict(n=255)):
        assert _fwd(native, p, **bad) == E, bad
    assert _fwd(native, _p(native, Hq=1 << 20, H=1, rows=1 << 11, at=8)) == native.SA_EUNSUPPORTED
    assert native.load_library().sparse_attn_paged_ws_bytes(ctypes.byref(p), None) == E


# ---- the Python layer

def test_python_layer_refuses_cpu_tensors_and_bad_kinds():
    torch = pytest.importorskip("torch")
    import block_sparse_routed_gb300 as bsr

    pages = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16)
    t, rs, kl = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsr.cache_write(x, x, pages, pages, t, rs, kl)
    with pytest.raises(ValueError):
        bsr.paged_attn(x, pages, pages, t, rs, kl)
    with pytest.raises(TypeError):
        bsr.cache_read(pages.float(), pages.float(), t, rs, kl, rows=1)
    with pytest.raises(ValueError):
        bsr.paged_cache(4, 1, page_size=48, device="cpu")
    with pytest.raises(ValueError):
        bsr.paged_cache(4, 1, dtype="int8", device="cpu")
    k, v, ke, ve = bsr.paged_cache(4, 2, page_size=16, dtype="e4m3", device="cpu")
    assert k.shape == v.shape == (4, 2, 16, 128) and k.dtype == torch.float8_e4m3fn
    assert ke.shape == ve.shape == (4, 2, 16) and ke.dtype == torch.uint8
