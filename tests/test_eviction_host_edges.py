"""Refusals of weights and eviction at their limits, without a GPU: outputs over
what a launch's blocks read, scales past what the factors hold."""

import ctypes

import pytest

from .test_eviction_host import E_FIELDS, _evict, _weigh
from .test_paged_host import _p, native  # noqa: F401

# seqs 3, H 2, keep 5; a table of 3 rows of 4 entries, 100 apart; addresses that no path here may touch
KL, TABLE, TO, KEPT, NEW = (k << 24 for k in range(1, 6))
SIZES = dict(seqs=3, H=2, pages=10, table_width=4, table_stride=100)
E = dict(E_FIELDS, keep=5, first=1, last=1, to_width=2, to_stride=50)
N_KEPT = 4 * 3 * 2 * 5  # bytes


def call(native, **kw):  # noqa: F811
    return _evict(native, _p(native, **SIZES), **{**dict(kl=KL, table=TABLE, to=TO, kept=KEPT, new=NEW, e=E), **kw})


@pytest.mark.parametrize("kw", [
    dict(new=KL), dict(new=KL + 4), dict(new=KL + 8), dict(new=KL - 4), dict(new=KL - 8),
    dict(kept=KL), dict(kept=KL + 8), dict(kept=KL - N_KEPT + 4),
    dict(new=KEPT), dict(new=KEPT + N_KEPT - 4), dict(new=KEPT - 8),
    dict(new=TABLE), dict(new=TABLE + 12), dict(new=TABLE - 8), dict(new=TABLE + 400 - 4), dict(new=TABLE + 812), dict(new=TABLE + 4 * 98),
    dict(kept=TABLE + 800 + 12), dict(kept=TABLE - N_KEPT + 4), dict(kept=TABLE + 16 + 400 - N_KEPT),
    dict(new=TO + 4), dict(new=TO + 400 + 4), dict(kept=TO + 200 - 4), dict(kept=TO - 4),
    dict(to=None, new=TABLE), dict(to=None, kept=KL),
])
def test_outputs_over_inputs_are_refused(native, kw):  # noqa: F811
    assert call(native, **kw) == native.SA_EINVAL


@pytest.mark.parametrize("kw", [
    dict(), dict(to=None), dict(new=KL + 12), dict(new=KL - 12), dict(kept=KL + 12), dict(kept=KL - N_KEPT),
    dict(new=KEPT + N_KEPT), dict(new=KEPT - 12),
    dict(new=TABLE + 16), dict(new=TABLE + 400 - 12), dict(new=TABLE + 816), dict(new=TABLE - 12),  # between a table's rows, too
    dict(kept=TABLE + 16), dict(kept=TABLE + 816), dict(kept=TABLE - N_KEPT), dict(kept=TO + 8), dict(kept=TO + 208), dict(new=TO + 408),
])
def test_outputs_beside_inputs_are_not(native, kw):  # noqa: F811
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses are nobody's")
    assert call(native, **kw) != native.SA_EINVAL  # (but there is no device)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("e,fine", [(-101, False), (-100, True), (60, True), (61, False), (99, False), (120, False)])
def test_scales(native, kind, e, fine):  # noqa: F811
    p, out = _p(native, kind=kind, scale=2.0 ** e), ctypes.c_uint64()
    want = native.SA_OK if fine else native.SA_EUNSUPPORTED
    assert native.load_library().sparse_attn_weigh_ws_bytes(ctypes.byref(p), ctypes.byref(out)) == want
    if not fine:
        assert _weigh(native, p) == want
