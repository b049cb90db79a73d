"""The paged cache where it can go wrong: calls that give up, values that are
not finite, the ends of the formats' ranges, arguments and streams.

Tolerances are those of ``tests/test_gpu_paged.py``; what differs is said at
the test.
"""

import math

import numpy as np
import pytest

import oracle as O
from oracle import paged as OP
from tests.test_gpu_paged import U, Batch, bits, run_attention

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def bsr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_routed_gb300 as m

    m.load_library()
    return m


KINDS = pytest.mark.parametrize("kind", ["bf16", "e4m3"])


# ---- calls that give up

@KINDS
@pytest.mark.parametrize("lens,news,H,Hq", [
    ([40], [1], 1, 4),              # one stage: every load is issued before anyone has looked
    ([64, 130, 1], [1, 1, 1], 2, 8),
    ([150], [3], 1, 4),             # 12 packed rows
    ([70], [60], 1, 2),             # one key tile
    ([300], [200], 1, 2),           # parts of no more tiles than the ring has slots
    ([300, 777, 20], [200, 140, 20], 2, 6),
])
def test_copies_in_flight_of_a_call_that_gives_up(bsr, kind, lens, news, H, Hq):
    """A producer that has issued all its loads when another warp's wait fails:
    the call reports the timeout, its copies land before its blocks end, and
    what runs next on the same multiprocessors finds its shared memory its own."""
    from block_sparse_routed_gb300 import _native

    b = Batch(lens, news, H, 64, kind, seed=2)
    q, o, lse = run_attention(bsr, b, Hq)
    ws = bsr.paged_workspace(q, b.k_pages, b.table, max(news))
    statuses = []
    for _ in range(20):
        prev = _native.sparse_attn_set_single_probe_waits(True)
        try:
            bsr.paged_attn(q, *b.where, max_new=max(news), **b.exps, ws=ws)
        finally:
            _native.sparse_attn_set_single_probe_waits(bool(prev))
        statuses.append(bsr.sparse_attn_last_device_status(ws))
        o2, l2 = bsr.paged_attn(q, *b.where, max_new=max(news), **b.exps, ws=ws)
        assert bsr.sparse_attn_last_device_status(ws) == 0
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert bsr.SA_ETIMEOUT in statuses
