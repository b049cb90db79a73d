"""Shared prefixes where a batch has empty slots, and what the device reports."""

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from .test_gpu_paged import Batch, bsr, check_attention  # noqa: E402,F401
from .test_gpu_prefix import i32, run_prefix, shared_batch  # noqa: E402


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


def two_forms(bsr, q, b):
    """Prefixes by the form for chunks, own keys by that for few rows: two workspaces in one."""
    size = lambda max_new: bsr.prefix_ws_bytes(q, b.k_pages, b.table, b.groups[0], max_new)  # noqa: E731
    return size(3) > size(None)


@pytest.mark.parametrize("bad", ["shared page", "own page", "group", "prefix", "length", "nothing"])
def test_either_part_reports(bsr, bad):
    """Where the two parts are different kernels, each with a status of its own."""
    b = shared_batch([100, 300, 80], [3, 3, 2], [0, 3], [640], 2, 64, "e4m3", seed=7)
    q = torch.randn((b.rows, 10, 128), device="cuda").bfloat16()
    assert two_forms(bsr, q, b)
    table, kl, (gs, pl) = b.table.clone(), b.kv_len.clone(), [t.clone() for t in b.groups]
    if bad == "shared page":
        table[0, 4] = b.pages  # (of the others' rows nobody looks at it)
    elif bad == "own page":
        table[1, 12] = -1
    elif bad == "group":
        gs[1] = 4
    elif bad == "prefix":
        pl[0] = -1
    elif bad == "length":
        kl[2] = 1 << 20
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, gs, 3)
    for _ in range(2):
        bsr.prefix_attn(q, b.k_pages, b.v_pages, table, b.row_start, kl, gs, pl, max_new=3, **b.exps, ws=ws)
        assert bsr.sparse_attn_last_device_status(ws) == (bsr.SA_OK if bad == "nothing" else bsr.SA_EINVAL)
    bsr.prefix_attn(q, *b.where, *b.groups, max_new=3, **b.exps, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_OK


def test_a_wait_that_gives_up_in_two_forms(bsr):
    from block_sparse_routed_gb300 import _native

    b = shared_batch([1000, 3000, 80], [3, 3, 2], [0, 3], [2000], 2, 64, "e4m3", seed=7)
    q, o, lse = run_prefix(bsr, b, 10)
    assert two_forms(bsr, q, b)
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, b.groups[0], 3)
    prev = _native.sparse_attn_set_single_probe_waits(True)
    try:
        statuses = []
        for _ in range(5):  # a single probe almost surely comes too early
            bsr.prefix_attn(q, *b.where, *b.groups, max_new=3, **b.exps, ws=ws)
            statuses.append(bsr.sparse_attn_last_device_status(ws))
            if statuses[-1] == bsr.SA_ETIMEOUT:
                break
    finally:
        _native.sparse_attn_set_single_probe_waits(bool(prev))
    assert bsr.SA_ETIMEOUT in statuses
    o2, l2 = bsr.prefix_attn(q, *b.where, *b.groups, max_new=3, **b.exps, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 60])
@pytest.mark.parametrize("bad", [([0, 3, 2], [64, 64]), ([0, 4], [64]), ([0, 3], [192]), ([-1, 2], [64])])
def test_valid_calls_after_bad_groups(bsr, kind, news, bad):
    b = Batch([200, 192 + news - 1, 300], [news, news, 1], 2, 64, kind, seed=4)
    q = torch.randn((b.rows, 16, 128), device="cuda").bfloat16()
    gs, pl = i32(*bad[0]), i32(*bad[1])
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, gs, news)
    bsr.prefix_attn(q, *b.where, gs, pl, max_new=news, **b.exps, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL
    gs, pl = i32(0, 3), i32(0)
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, gs, news)
    o, lse = bsr.prefix_attn(q, *b.where, gs, pl, max_new=news, **b.exps, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_OK
    check_attention(b, q, o, lse)


@pytest.mark.parametrize("groups,prefix", [([0, 4], [64]), ([3, 1], [64]), ([0, 1], [-5]), ([0, 1], [64])])
def test_one_sequence_shares_nothing(bsr, groups, prefix):
    """Its groups are not looked at: the call is paged_attn's, bit for bit."""
    b = Batch([200], [5], 2, 64, seed=4)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    gs, pl = i32(*groups), i32(*prefix)
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, gs)
    o, lse = bsr.prefix_attn(q, *b.where, gs, pl, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_OK
    o2, lse2 = bsr.paged_attn(q, *b.where)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
