"""Calls of the routed attention that end early, many times in turn with good
ones: what a block of a given-up or refused call had in flight (copies into its
shared memory, products, stores to tensor memory) must not reach the next
block on its multiprocessor.  The failures are made as in
``tests/test_gpu_failure.py``."""

import pytest

from tests.test_gpu_failure import _corrupt_cases, _fwd, setup  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_calls_that_give_up_in_turn_with_good_ones(setup):  # noqa: F811
    s = setup
    native, bsr = s["native"], s["bsr"]
    statuses = []
    for _ in range(20):
        prev = native.sparse_attn_set_single_probe_waits(True)
        try:
            _, st = _fwd(s)
        finally:
            native.sparse_attn_set_single_probe_waits(bool(prev))
        statuses.append(st)
        o, st = _fwd(s)
        assert st == bsr.SA_OK and torch.equal(o, s["o_ref"])
    assert bsr.SA_ETIMEOUT in statuses


def test_refused_lists_in_turn_with_good_ones(setup):  # noqa: F811
    s = setup
    bsr = s["bsr"]
    for idx, cnt in _corrupt_cases(s).values():
        idx, cnt = (torch.from_numpy(x.copy()).cuda() for x in (idx, cnt))
        for _ in range(5):
            _, st = _fwd(s, idx.reshape(s["idx"].shape), cnt.reshape(s["cnt"].shape))
            assert st == bsr.SA_EINVAL
            o, st = _fwd(s)
            assert st == bsr.SA_OK and torch.equal(o, s["o_ref"])
