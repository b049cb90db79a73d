"""Attention where groups of sequences share a prefix, against the fp64 oracle
of each sequence alone.  Tolerances are those of the paged attention: a row's
result is still one softmax, joined from one part more."""

import math

import numpy as np
import pytest

from oracle import paged as OP

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from .test_gpu_paged import U, Batch, bsr, check_attention, rows_of  # noqa: E402,F401


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def shared_batch(own, news, groups, prefixes, H, page, kind, seed=0, **kw):
    """own: tokens of each sequence behind the whole pages that it shares;
    groups: first sequences; prefixes: tokens of each group."""
    pages = [0] * len(own)
    for g, p in enumerate(prefixes):
        for s in range(groups[g], groups[g + 1]):
            pages[s] = p // page
    b = Batch([n + p * page for n, p in zip(own, pages)], news, H, page, kind, seed=seed, **kw)
    for g in range(len(prefixes)):
        for s in range(groups[g] + 1, groups[g + 1]):
            b.table_np[s, :pages[s]] = b.table_np[groups[g], :pages[s]]
    b.table = torch.from_numpy(b.table_np).cuda()
    b.groups = i32(*groups), i32(*prefixes)
    return b


def run_prefix(bsr, b, Hq, seed=1, tight=True, q=None, **kw):
    g = torch.Generator().manual_seed(seed)
    if q is None:
        q = torch.randn((b.rows, Hq, 128), generator=g).bfloat16().cuda() * 2
    o = torch.full((b.rows, Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.rows, Hq), 3.0, device="cuda")
    max_new = max(b.news) if tight else None
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, b.groups[0], max_new)
    ws.fill_(255)  # scratch is the call's own business
    bsr.prefix_attn(q, *b.where, *b.groups, max_new=max_new, **b.exps, o=o, lse=lse, ws=ws, **kw)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    return q, o, lse


CASES = [
    # own, news, groups, prefixes, H, Hq, page, causal
    ([5, 9], [1, 1], [0, 2], [64], 2, 8, 64, True),
    ([5, 9], [1, 1], [0, 2], [63], 2, 8, 64, True),                  # not one whole page is shared
    ([70, 1, 200], [1, 1, 1], [0, 3], [500], 1, 40, 16, True),
    ([70, 1, 200], [1, 1, 1], [0, 3], [500], 1, 40, 16, False),
    ([70, 20, 200, 33, 5], [1, 4, 30, 2, 5], [0, 2, 3, 5], [500, 300, 0], 2, 6, 32, True),   # a group of one; no prefix
    ([70, 20, 200, 33, 5], [1, 4, 30, 2, 5], [1, 3, 5], [129, 1000], 2, 6, 32, True),        # a sequence of no group
    ([70, 20, 200, 33, 5], [1, 4, 30, 2, 5], [0, 0, 2, 2, 4], [77, 200, 300, 140], 3, 3, 128, False),  # empty groups
    ([0, 64, 0], [0, 64, 0], [0, 3], [256], 1, 2, 64, True),         # sequences without rows
    ([264, 264, 264], [264, 264, 264], [0, 3], [330], 2, 2, 64, False),
    ([300, 150], [300, 90], [0, 2], [700], 1, 7, 128, True),
    ([17, 33], [2, 3], [0, 2], [90], 1, 300, 16, True),              # a token is more than a tile of rows
    ([3, 2, 40], [6, 9, 1], [0, 2, 3], [10, 32], 2, 4, 16, True),    # more rows than tokens, where nothing is shared
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tight", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_prefixes(bsr, kind, tight, case):
    own, news, groups, prefixes, H, Hq, page, causal = CASES[case]
    b = shared_batch(own, news, groups, prefixes, H, page, kind, seed=case, first_row=1, after=2)
    q, o, lse = run_prefix(bsr, b, Hq, tight=tight, causal=causal)
    check_attention(b, q, o, lse, causal, filled=3.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 3, 40])
def test_a_long_prefix_is_split_and_joined(bsr, kind, news):
    b = shared_batch([900, 50, 64], [news, 1, news], [0, 3], [9505], 2, 64, kind, seed=5)
    q, o, lse = run_prefix(bsr, b, 10)
    check_attention(b, q, o, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_sequences_and_groups(bsr, kind):
    g = np.random.default_rng(5)
    own = [int(x) for x in g.integers(3, 40, 700)]
    news = [int(g.integers(0, 4)) if g.random() < 0.4 else 0 for _ in own]
    groups = sorted(int(x) for x in g.choice(700, 120, replace=False)) + [699]
    prefixes = [int(x) for x in g.integers(0, 90, 120)]
    b = shared_batch(own, news, groups, prefixes, 1, 16, kind, seed=6)
    q, o, lse = run_prefix(bsr, b, 4)
    check_attention(b, q, o, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 60])
def test_the_same_as_without_sharing(bsr, kind, news):
    """Up to the order of sums: against the oracle both, and the differences small."""
    b = shared_batch([100, 300, 77, 61], [news] * 4, [0, 2, 4], [640, 200], 2, 64, kind, seed=7)
    q, o, lse = run_prefix(bsr, b, 8, scale=0.05)
    o2, lse2 = bsr.paged_attn(q, *b.where, scale=0.05, **b.exps)
    check_attention(b, q, o, lse, scale=0.05)
    check_attention(b, q, o2, lse2, scale=0.05)


def test_strided_queries_and_other_streams(bsr):
    b = shared_batch([100, 300], [1, 70], [0, 2], [640], 2, 64, "bf16", seed=7)
    x = torch.randn((b.rows, 3, 4, 136), device="cuda").bfloat16()
    q, o, lse = run_prefix(bsr, b, 4, q=x[:, 1, :, :128])
    check_attention(b, q, o, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = bsr.prefix_attn(q, *b.where, *b.groups, max_new=70, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_odd_values_reach_only_the_rows_that_see_them(bsr, kind):
    """NaN in the prefix reaches its group's rows alone; in own tokens, the rows
    behind them."""
    b = shared_batch([40, 50, 60, 70], [20, 30, 1, 40], [0, 2, 4], [128, 192], 2, 64, kind, seed=3)
    q, o, lse = run_prefix(bsr, b, 4)
    spoil = [(0, 100, [0, 1]), (3, 192 + 45, [3])]  # (sequence, token, sequences that see it)
    for s, j, who in spoil:
        v = b.v_pages.clone()
        ve = None if b.v_exp is None else b.v_exp.clone()
        if kind == "bf16":
            v[b.table_np[s, j // 64], :, j % 64, 3] = math.nan
        else:
            ve[b.table_np[s, j // 64], :, j % 64] = 255
        o2, lse2 = bsr.prefix_attn(q, b.k_pages, v, *b.where[2:], *b.groups, max_new=40, k_exp=b.k_exp, v_exp=ve)
        assert torch.equal(lse, lse2)
        for t in range(4):
            rows = [(r, p) for r, p in OP.positions(b.starts, b.lens, t)]
            for r, p in rows:
                sees = t in who and p >= j
                assert bool(o2[r, :, 3].isnan().all()) == sees and bool(o2[r].isnan().any()) == sees, (t, r, p)
                if not sees:
                    assert torch.equal(o2[r], o[r])


def test_bitwise_repeatable_and_captured(bsr):
    b = shared_batch([900, 50, 64], [1, 1, 3], [0, 3], [4000], 2, 64, "e4m3", seed=5)
    q, o, lse = run_prefix(bsr, b, 10)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, b.groups[0], 3)
    step = lambda: bsr.prefix_attn(q, *b.where, *b.groups, max_new=3, **b.exps, o=o2, lse=lse2, ws=ws)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        o2.zero_()
        graph.replay()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # lengths and groups are read when it runs
    b.groups[1].fill_(0)
    graph.replay()
    assert bsr.sparse_attn_last_device_status(ws) == 0
    check_attention(b, q, o2, lse2)


@pytest.mark.parametrize("groups,prefixes", [
    ([0, 3, 2], [64, 64]),        # not ascending
    ([-1, 2], [64]),
    ([0, 4], [64]),               # past the sequences
    ([0, 3], [-1]),
    ([0, 3], [1 << 20]),          # more than the table has pages for
    ([0, 3], [192]),              # rows inside the prefix
])
@pytest.mark.parametrize("news", [1, 40])
def test_bad_groups_are_reported(bsr, groups, prefixes, news):
    b = Batch([200, 192 + news - 1, 300], [news, news, 1], 2, 64, seed=4)
    q = torch.randn((b.rows, 16, 128), device="cuda").bfloat16()
    gs, pl = i32(*groups), i32(*prefixes)
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, gs, news)
    bsr.prefix_attn(q, *b.where, gs, pl, max_new=news, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL
    bsr.prefix_attn(q, *b.where, i32(0, 3), i32(0), max_new=news, ws=bsr.prefix_workspace(q, b.k_pages, b.table, gs, news))
    bad = b.table.clone()
    bad[0, 1] = b.pages
    gs = i32(0, 3)
    ws = bsr.prefix_workspace(q, b.k_pages, bad, gs, news)
    bsr.prefix_attn(q, b.k_pages, b.v_pages, bad, b.row_start, b.kv_len, gs, i32(128), max_new=news, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_wait_that_gives_up_is_reported(bsr, kind):
    from block_sparse_routed_gb300 import _native

    b = shared_batch([100, 300], [1, 70], [0, 2], [2000], 2, 64, kind, seed=7)
    q, o, lse = run_prefix(bsr, b, 4)
    ws = bsr.prefix_workspace(q, b.k_pages, b.table, b.groups[0], 70)
    prev = _native.sparse_attn_set_single_probe_waits(True)
    try:
        statuses = []
        for _ in range(5):  # a single probe almost surely comes too early
            bsr.prefix_attn(q, *b.where, *b.groups, max_new=70, **b.exps, ws=ws)
            statuses.append(bsr.sparse_attn_last_device_status(ws))
            if statuses[-1] == bsr.SA_ETIMEOUT:
                break
    finally:
        _native.sparse_attn_set_single_probe_waits(bool(prev))
    assert bsr.SA_ETIMEOUT in statuses
    o2, l2 = bsr.prefix_attn(q, *b.where, *b.groups, max_new=70, **b.exps, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_nothing_to_do(bsr):
    k, v, _, _ = bsr.paged_cache(4, 2, 16)
    empty = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    for seqs in (0, 3):
        batch = (torch.empty((seqs, 2), dtype=torch.int32, device="cuda"), i32(*[0] * (seqs + 1)), i32(*[0] * seqs))
        for gs, pl in ((i32(0), i32()), (i32(0, seqs), i32(0))):
            ws = bsr.prefix_workspace(empty, k, batch[0], gs).fill_(255)
            o, lse = bsr.prefix_attn(empty, k, v, *batch, gs, pl, ws=ws)
            assert o.shape == (0, 4, 128) and bsr.sparse_attn_last_device_status(ws) == 0
    # rows, but of no sequence
    q = torch.ones((3, 4, 128), dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 5.0)
    bsr.prefix_attn(q, k, v, torch.zeros((2, 2), dtype=torch.int32, device="cuda"), i32(0, 0, 0), i32(0, 0), i32(0, 2), i32(0), o=o)
    assert (o == 5).all()


def test_refusals_of_the_python_layer(bsr):
    b = shared_batch([100, 300], [1, 1], [0, 2], [64], 2, 64, "bf16", seed=7)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    gs, pl = b.groups
    call = lambda q=q, gs=gs, pl=pl, **kw: bsr.prefix_attn(q, *b.where, gs, pl, **kw)  # noqa: E731
    for bad in (dict(q=q[:, :3]), dict(q=q.half()), dict(q=q.cpu()), dict(gs=gs.long()), dict(pl=pl.long()), dict(gs=gs[:1]),
                dict(pl=i32(1, 2)), dict(gs=gs.cpu()), dict(gs=gs[None]), dict(gs=i32(0, 9, 2)[::2]), dict(max_new=-1),
                dict(o=torch.empty((b.rows, 4, 64), dtype=torch.bfloat16, device="cuda")), dict(k_exp=gs),
                dict(lse=torch.empty((b.rows, 4), dtype=torch.float64, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    with pytest.raises(bsr.SparseAttnError):
        call(scale=-1.0)
    with pytest.raises(bsr.SparseAttnError):
        call(ws=bsr.paged_workspace(q, b.k_pages, b.table, 1)[:256])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_one_prompt_many_answers(bsr, kind):
    """A prompt is written once; answers grow behind it, attending by
    prefix_attn, and are cut back by what their own tokens received."""
    H, Hq, page, P, S, budget = 2, 8, 16, 100, 5, 140
    whole = P // page
    per = 5
    k, v, ke, ve = bsr.paged_cache(whole + S * per, H, page, kind)
    exps = dict(k_exp=ke, v_exp=ve)
    w = bsr.cache_weights(k)
    g = torch.Generator().manual_seed(0)
    perm = torch.randperm(whole + S * per, generator=g).to(torch.int32)
    table = torch.cat([perm[:whole].repeat(S, 1), perm[whole:].reshape(S, per)], 1).cuda()
    xk, xv = rows_of(P, H, seed=3)
    for s in range(S):  # (the page that the prompt ends in is each answer's own)
        bsr.cache_write(xk, xv, k, v, table[s:s + 1], i32(0, P), i32(P), **exps)
    rs, kl = i32(*range(S + 1)), i32(*[P] * S)
    gs, pl = i32(0, S), i32(P)
    hist = [[t.double().cpu().numpy() for t in bsr.cache_read(k, v, table[:1], i32(0, P), i32(P), rows=P, **exps)] for _ in range(S)]
    hist = [[[(a[j, h], c[j, h]) for j in range(P)] for h in range(H)] for a, c in hist]
    for step in range(70):
        nk, nv = (torch.randn((S, H, 128), generator=g).bfloat16().cuda() for _ in range(2))
        q = (torch.randn((S, Hq, 128), generator=g) * 2).bfloat16().cuda()
        kl.add_(1)
        bsr.cache_write(nk, nv, k, v, table, rs, kl, **exps)
        o, lse = bsr.prefix_attn(q, k, v, table, rs, kl, gs, pl, max_new=1, **exps)
        bsr.cache_weigh(q, lse, w, k, table, rs, kl, max_new=1, first=P, k_exp=ke)
        back = [t.double().cpu().numpy() for t in bsr.cache_read(k, v, table, rs, kl, rows=S, **exps)]
        n, q64 = int(kl[0]), q.double().cpu().numpy()
        for s in range(S):
            for h in range(H):
                hist[s][h].append((back[0][s, h], back[1][s, h]))
                if step % 10 in (0, 9):
                    kk, vv = (np.stack([t[x] for t in hist[s][h]])[:, None] for x in range(2))
                    heads = slice(4 * h, 4 * h + 4)
                    ro, rl, mass, reach = OP.paged_attention(q64[s:s + 1, heads], kk, vv, [n - 1], n)
                    ds = 264 * U * reach
                    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (n + 64) * U)[..., None] * mass
                    assert np.all(np.abs(o[s:s + 1, heads].double().cpu().numpy() - ro) <= tol), step
        if n > budget:
            kept, new_len = bsr.cache_evict(k, v, w, table, kl, 120, first=P, last=4, **exps)
            kl.copy_(new_len)
            for s in range(S):
                for h in range(H):
                    mine = kept[s, h].tolist()
                    assert mine[:P] == list(range(P)) and mine[-4:] == list(range(n - 4, n))
                    hist[s][h] = [hist[s][h][j] for j in mine]
    assert int(kl[0]) < P + 70


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,H,group", [(1, 2, 17), (3, 2, 7), (4, 1, 6), (24, 2, 1), (3, 1, 8), (5, 1, 5), (1, 1, 33)])
@pytest.mark.parametrize("causal", [True, False])
def test_own_rows_around_a_tile(bsr, kind, news, H, group, causal):
    """17 to 24 rows of a sequence and key head (one tile in E4M3), fewer beside them, and one more."""
    b = shared_batch([300, 64, 31, 700, 90, 5], [news, news, 1, news, 0, 2], [0, 3, 6], [320, 64], H, 32, kind, seed=news + group, first_row=1, after=1)
    q, o, lse = run_prefix(bsr, b, H * group, causal=causal)
    check_attention(b, q, o, lse, causal, filled=3.0)
    q, o, lse = run_prefix(bsr, b, H * group, causal=causal, scale=2.5)
    check_attention(b, q, o, lse, causal, scale=2.5, filled=3.0)


@pytest.mark.parametrize("news,group", [(3, 7), (4, 6)])
def test_long_own_keys_of_a_tile(bsr, news, group):
    """Parts of a unit in many blocks."""
    b = shared_batch([4000, 77, 5200], [news, 1, news], [0, 2], [640], 2, 64, "e4m3", seed=9)
    q, o, lse = run_prefix(bsr, b, 2 * group)
    check_attention(b, q, o, lse)
