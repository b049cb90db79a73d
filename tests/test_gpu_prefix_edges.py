"""Shared prefixes where a batch has empty slots."""

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from .test_gpu_paged import bsr, check_attention  # noqa: E402,F401
from .test_gpu_prefix import run_prefix, shared_batch  # noqa: E402


def empty_slot(b, s, length):
    """A finished sequence: no rows, its length no longer the prefix's, its table row nobody's."""
    assert b.news[s] == 0
    b.lens[s] = length
    b.kv_len[s] = length
    b.table[s] = -7


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 3, 40])  # all rows by the form for few; E4M3: own keys by it; all by the form for chunks
@pytest.mark.parametrize("slots", [[(2, 0)], [(2, 100)], [(0, 0)], [(0, 0), (1, 0)], [(0, 5), (4, 0)], [(3, 0), (4, 63)]])
def test_empty_slots_in_a_group(bsr, kind, news, slots):
    """The prefix is read by the row of a sequence that has rows, wherever the group begins."""
    new = [news, news, 1, news, 1, 2]
    for s, _ in slots:
        new[s] = 0
    b = shared_batch([70, 90, 33, 120, 65, 40], new, [0, 5, 6], [330, 64], 2, 64, kind, seed=news, first_row=1, after=1)
    for s, n in slots:
        empty_slot(b, s, n)
    q, o, lse = run_prefix(bsr, b, 10)
    check_attention(b, q, o, lse, filled=3.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_group_of_empty_slots(bsr, kind):
    b = shared_batch([70, 90, 33, 50], [0, 0, 4, 2], [0, 2, 4], [330, 64], 2, 64, kind, seed=3, after=1)
    for s in (0, 1):
        empty_slot(b, s, 0)
    q, o, lse = run_prefix(bsr, b, 10)
    check_attention(b, q, o, lse, filled=3.0)
