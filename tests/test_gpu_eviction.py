"""Weights that cached keys receive, and eviction by them, against the fp64
oracle.

Weights (u = 2^-24).  With R = scale * sum_d |q_d k_d| of a row and a key:
  * the logit is an FP32 sum of 128 exact products in some order, each addition
    off by at most one step (2u) even where the tensor core truncates; scaling
    and the subtraction of lse in the exponent's base: 8u (R + |lse|) at most.
    Together at most (2 * 128 + 8) u (R + |lse|), relative to the term (first
    order, doubled below), and 2^-22 of ex2.
  * the sum of n terms and of what was there, in some order: (n + 8) u of it.
  * a term below 2^-126 may vanish.
Moves are compared bit for bit, and positions exactly.
"""

import math

import numpy as np
import pytest

from oracle import paged as OP

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from .test_gpu_paged import U, Batch, bsr, rows_of  # noqa: E402,F401


def fresh_weights(b, seed=0):
    g = np.random.default_rng(seed)
    w = np.exp(g.standard_normal((b.pages, b.H, b.page))).astype(np.float32)
    return torch.from_numpy(w).cuda()


def run_weigh(bsr, b, Hq, q=None, lse=None, first=0, accumulate=True, tight=True, check=True, seed=1, **kw):
    g = torch.Generator().manual_seed(seed)
    if q is None:
        q = torch.randn((b.rows, Hq, 128), generator=g).bfloat16().cuda() * 2
    max_new = max(b.news) if tight else None
    if lse is None:
        _, lse = bsr.paged_attn(q, *b.where, max_new=max_new, **b.exps, **kw)
    w = fresh_weights(b)
    before = w.cpu().numpy().copy()
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    out = bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len, max_new=max_new, first=first,
                          accumulate=accumulate, k_exp=b.k_exp, ws=ws, **kw)
    assert out is w
    assert bsr.sparse_attn_last_device_status(ws) == 0
    if check:
        check_weights(b, q, lse, before, w, first, accumulate, **kw)
    return q, lse, w


def check_weights(b, q, lse, before, w, first, accumulate, causal=True, window=0, scale=None):
    q64, l64, got = q.double().cpu().numpy(), lse.double().cpu().numpy(), w.cpu().numpy()
    want, tol = before.astype(np.float64), np.zeros_like(before, dtype=np.float64)
    for s, n in enumerate(b.lens):
        rows = [r for r, _ in OP.positions(b.starts, b.lens, s)]
        pos = [p for _, p in OP.positions(b.starts, b.lens, s)]
        if not rows or not n:
            continue
        k = OP.gather(b.k64, b.table_np, s, n)
        r, slack, count = OP.received(q64[rows], l64[rows], k, pos, n, causal, window, scale)
        for j in range(first, n):
            at = (b.table_np[s, j // b.page], slice(None), j % b.page)
            old = before[at].astype(np.float64) if accumulate and j < n - len(rows) else 0.0
            want[at] = old + r[:, j]
            tol[at] = (2 * (2 * 128 + 8) * U * slack[:, j] + 2.0 ** -21 * r[:, j]
                       + (count[:, j] + 8) * U * want[at] + count[:, j] * 2.0 ** -126)
            if accumulate:
                tol[at] = np.where(count[:, j] == 0, 0, tol[at])
    d = np.abs(got - want)
    assert np.all(np.isfinite(got))
    assert np.all(d <= tol), (d.max(), np.argwhere(d > tol)[:5], len(np.argwhere(d > tol)))


RAGGED = ([1, 0, 63, 64, 65, 200, 129], [1, 0, 1, 1, 1, 1, 1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hq", [(1, 1), (2, 16), (8, 8), (3, 15), (1, 40)])
def test_weights_of_single_tokens(bsr, kind, page, H, Hq):
    b = Batch(*RAGGED, H, page, kind, seed=H + Hq, after=2)
    run_weigh(bsr, b, Hq)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,news,H,Hq,page,causal,window", [
    ([300, 77, 5], [4, 2, 5], 2, 6, 64, True, 0),
    ([300, 77, 5], [4, 2, 5], 2, 6, 64, False, 0),
    ([300, 700, 5, 0], [4, 3, 5, 2], 1, 8, 16, True, 37),     # windows end inside pages; rows without a token
    ([3, 2], [6, 9], 2, 4, 16, True, 0),                      # more rows than tokens
    ([3, 2], [6, 9], 2, 4, 16, False, 0),
    ([130], [130], 1, 1, 64, True, 0),
    ([260, 1, 90], [200, 1, 33], 2, 10, 32, True, 0),
    ([260, 1, 90], [200, 1, 33], 2, 10, 32, False, 0),
    ([513, 520], [129, 257], 1, 3, 128, True, 100),
    ([700], [300], 3, 21, 64, True, 0),
    ([600], [600], 1, 2, 16, True, 1),                        # every row sees itself alone
    ([400, 17], [20, 3], 1, 40, 64, True, 0),
    ([90, 170], [2, 3], 1, 300, 64, True, 0),                 # a token is more than a tile of rows
])
@pytest.mark.parametrize("first,accumulate,tight", [(0, True, True), (4, False, True), (70, True, False)])
def test_weights_of_chunks(bsr, kind, lens, news, H, Hq, page, causal, window, first, accumulate, tight):
    b = Batch(lens, news, H, page, kind, seed=len(lens) + window, first_row=1, after=1)
    run_weigh(bsr, b, Hq, first=first, accumulate=accumulate, tight=tight, causal=causal, window=window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,Hq", [(1, 4), (150, 4), (33, 14)])
def test_weights_of_a_long_context(bsr, kind, news, Hq):
    b = Batch([9505, 40], [news, 1], 2, 64, kind, seed=5)
    run_weigh(bsr, b, Hq)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,news,H,Hq,window", [([2600], [40], 24, 24, 0),        # many units a block, one step each
                                                   ([5200], [700], 8, 24, 0),        # many, of many steps
                                                   ([3000, 2000], [900, 1], 6, 30, 1000)])
def test_weights_of_many_units(bsr, kind, lens, news, H, Hq, window):
    b = Batch(lens, news, H, 64, kind, seed=15)
    q, lse, w = run_weigh(bsr, b, Hq, window=window, check=False)
    # a few keys of a few heads
    before = fresh_weights(b).cpu().numpy()
    q64, l64, got = q.double().cpu().numpy(), lse.double().cpu().numpy(), w.cpu().numpy()
    g = Hq // H
    for s, n in enumerate(lens):
        rows = [r for r, _ in OP.positions(b.starts, lens, s)]
        pos = [p for _, p in OP.positions(b.starts, lens, s)]
        k = OP.gather(b.k64, b.table_np, s, n)
        for h in (0, H // 2, H - 1):
            r, slack, count = OP.received(q64[rows][:, h * g:(h + 1) * g], l64[rows][:, h * g:(h + 1) * g], k[:, h:h + 1], pos, n,
                                          True, window)
            j = np.arange(n)
            at = (b.table_np[s, j // 64], h, j % 64)
            want = np.where(j < n - len(rows), before[at], 0) + r[0]
            tol = 2 * 264 * U * slack[0] + 2.0 ** -21 * r[0] + (count[0] + 8) * U * want + count[0] * 2.0 ** -126
            assert np.all(np.abs(got[at] - want) <= tol), (s, h)


def test_weights_of_strided_queries_and_scales(bsr):
    b = Batch([200, 90], [70, 1], 2, 64, seed=4)
    x = torch.randn((b.rows, 3, 4, 136), device="cuda").bfloat16()
    run_weigh(bsr, b, 4, q=x[:, 1, :, :128], scale=0.3)
    same = torch.randn((1, 1, 128), device="cuda").bfloat16().expand(b.rows, 4, 128)
    run_weigh(bsr, b, 4, q=same)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 60])
def test_many_sequences_are_weighed(bsr, kind, news):
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(0, 40, 1100)]
    rows = [int(g.integers(0, news + 1)) if g.random() < 0.3 else 0 for _ in lens]
    rows[700] = news
    b = Batch(lens, rows, 1, 16, kind, seed=6)
    run_weigh(bsr, b, 4)


@pytest.mark.parametrize("news", [1, 60])
def test_rows_without_a_sum_count_nothing(bsr, news):
    """lse = -inf (a row that saw no key) and +inf."""
    b = Batch([300, 90], [news, 1], 2, 64, seed=4)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    _, lse = bsr.paged_attn(q, *b.where)
    lse[0, 1], lse[b.rows - 1, 3] = -math.inf, math.inf
    w = fresh_weights(b)
    before = w.cpu().numpy().copy()
    bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len)
    lse[lse == math.inf] = -math.inf  # to the oracle: no such row
    check_weights(b, q, lse, before, w, 0, True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [3, 60])
def test_a_key_that_is_nan_spoils_its_own_weight_only(bsr, kind, news):
    b = Batch([300, 90], [news, 1], 2, 64, kind, seed=4)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    _, lse = bsr.paged_attn(q, *b.where, **b.exps)
    clean = fresh_weights(b)
    bsr.cache_weigh(q, lse, clean, b.k_pages, b.table, b.row_start, b.kv_len, k_exp=b.k_exp)
    pg, sl = b.table_np[0, 2], 7  # token 135
    if kind == "bf16":
        b.k_pages[pg, 1, sl, 5] = math.nan
    else:
        b.k_exp[pg, 1, sl] = 255
    w = fresh_weights(b)
    bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len, k_exp=b.k_exp)
    assert w[pg, 1, sl].isnan()
    w[pg, 1, sl] = clean[pg, 1, sl]
    assert torch.equal(w, clean)


def test_weights_sum_to_the_rows(bsr):
    """Each row gives each key head as much as the group has query heads."""
    for news in (1, 90):
        b = Batch([1000, 333], [news, 1], 2, 64, seed=2)
        q = torch.randn((b.rows, 8, 128), device="cuda").bfloat16()
        _, lse = bsr.paged_attn(q, *b.where)
        w = bsr.cache_weights(b.k_pages)
        bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len, accumulate=False)
        for h in range(2):
            assert math.isclose(w[:, h].double().sum().item(), 4 * b.rows, rel_tol=1e-4)


def test_weigh_is_repeatable_and_goes_by_its_stream(bsr):
    b = Batch([3000, 70], [40, 1], 2, 64, "e4m3", seed=9)
    q, lse, w = run_weigh(bsr, b, 8)
    side = torch.cuda.Stream()
    for stream in (None, side):
        w2 = fresh_weights(b)
        side.wait_stream(torch.cuda.current_stream())
        bsr.cache_weigh(q, lse, w2, b.k_pages, b.table, b.row_start, b.kv_len, max_new=40, k_exp=b.k_exp, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(w, w2)


# ---- eviction

def evict_case(lens, H, page, kind, seed=0, ties=False):
    b = Batch(lens, [0] * len(lens), H, page, kind, seed=seed, spare=2)
    g = np.random.default_rng(seed + 1)
    w = np.exp(2 * g.standard_normal((b.pages, H, page))).astype(np.float32)
    if ties:
        w = np.round(w)
    w[g.random(w.shape) < 0.3] = 0.0
    return b, w


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy().copy()


def run_evict(bsr, b, w, keep, first=0, last=0, to=False, **kw):
    """Runs the call and checks every byte of cache and weights."""
    H, page = b.H, b.page
    parts = [b.k_pages, b.v_pages] + ([b.k_exp, b.v_exp] if b.k_exp is not None else [])
    to_np = None
    if to:  # pages behind the pool's own
        more = -(-keep // page)
        extra = len(b.lens) * more
        g = np.random.default_rng(3)
        to_np = (b.pages + g.permutation(extra)).astype(np.int32).reshape(len(b.lens), more)
        parts = [torch.cat([t.view(torch.uint8), torch.full((extra, *t.view(torch.uint8).shape[1:]), 77, dtype=torch.uint8, device="cuda")]).view(t.dtype)
                 for t in parts]
        w = np.concatenate([w, np.full((extra, H, page), 5.0, dtype=np.float32)])
    wt = torch.from_numpy(w).cuda()
    want = [raw(t).reshape(t.shape[0], H, page, -1) for t in parts] + [w.copy()[..., None]]
    src = [x.copy() for x in want]
    want_kept = np.full((len(b.lens), H, keep), -1, dtype=np.int32)
    for s, n in enumerate(b.lens):
        for h in range(H):
            j = np.arange(n)
            mine = w[b.table_np[s, j // page], h, j % page]
            kept = OP.survivors(mine, keep, first, last)
            want_kept[s, h, :len(kept)] = kept
            dst = b.table_np[s] if to_np is None else to_np[s]
            for i, p in enumerate(kept):
                for x, y in zip(want, src):
                    x[dst[i // page], h, i % page] = y[b.table_np[s, p // page], h, p % page]
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    exps = dict(k_exp=parts[2], v_exp=parts[3]) if len(parts) > 2 else {}
    kept, new_len = bsr.cache_evict(parts[0], parts[1], wt, b.table, b.kv_len, keep, first=first, last=last,
                                    to_table=None if to_np is None else torch.from_numpy(to_np).cuda(), ws=ws, **exps, **kw)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert new_len.tolist() == [min(n, keep) for n in b.lens]
    for t, x in zip(parts + [wt], want):
        assert np.array_equal(raw(t), x.view(np.uint8).reshape(raw(t).shape))
    return kept, new_len


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("to", [False, True])
@pytest.mark.parametrize("lens,H,page,keep,first,last", [
    ([100], 1, 16, 37, 0, 0),
    ([100, 0, 37, 38, 1, 36], 3, 16, 37, 4, 5),        # at, below and above the budget; none
    ([257, 300], 2, 128, 1, 0, 0),                     # one token stays
    ([257, 300], 2, 64, 1, 1, 0),
    ([257, 300], 2, 64, 40, 15, 25),                   # nothing to choose
    ([257, 300], 2, 32, 256, 0, 255),                  # one goes, one stays by weight
    ([1500, 40, 900], 2, 64, 700, 4, 64),
    ([2100], 8, 32, 1500, 33, 100),
])
def test_eviction(bsr, kind, to, lens, H, page, keep, first, last):
    b, w = evict_case(lens, H, page, kind, seed=len(lens) + keep)
    run_evict(bsr, b, w, keep, first, last, to)


@pytest.mark.parametrize("kind,to", [("bf16", False), ("e4m3", True), ("e4m3", False)])
def test_eviction_of_a_long_context(bsr, kind, to):
    b, w = evict_case([9505, 3000], 2, 64, kind, seed=7)
    run_evict(bsr, b, w, 5000, 4, 500, to)


def test_eviction_past_shared_memory(bsr):
    """More tokens than the selection keeps in shared memory."""
    b, w = evict_case([70001], 1, 128, "e4m3", seed=7)
    run_evict(bsr, b, w, 30000, 4, 500)


def test_eviction_of_many_sequences(bsr):
    g = np.random.default_rng(2)
    b, w = evict_case([int(x) for x in g.integers(0, 90, 700)], 2, 16, "bf16", seed=3)
    run_evict(bsr, b, w, 40, 3, 9)


@pytest.mark.parametrize("to", [False, True])
def test_ties_and_odd_weights(bsr, to):
    """Equal weights go to the earlier token; infinities, both zeros, negative
    weights and NaN have their places."""
    b, w = evict_case([600, 500], 2, 64, "bf16", seed=5, ties=True)
    run_evict(bsr, b, w, 200, 2, 10, to)
    run_evict(bsr, b, np.zeros_like(w), 200, 2, 10, to)
    g = np.random.default_rng(1)
    w = g.choice(np.array([0.0, -0.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-45, -1e-45], dtype=np.float32), w.shape)
    w.view(np.uint32)[np.isnan(w) & (g.random(w.shape) < 0.5)] |= 0x80000000
    run_evict(bsr, b, w, 200, 2, 10, to)


def test_nothing_to_evict(bsr):
    k, v, _, _ = bsr.paged_cache(4, 2, 16)
    w = bsr.cache_weights(k)
    i32 = dict(dtype=torch.int32, device="cuda")
    kept, new_len = bsr.cache_evict(k, v, w, torch.empty((0, 2), **i32), torch.zeros(0, **i32), 5)
    assert kept.shape == (0, 2, 5) and new_len.shape == (0,)
    kept, new_len = bsr.cache_evict(k, v, w, torch.zeros((3, 0), **i32), torch.zeros(3, **i32), 5)
    assert (kept == -1).all() and not new_len.any()
    empty = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    bsr.cache_weigh(empty, torch.empty((0, 4), device="cuda"), w, k, torch.zeros((3, 0), **i32), torch.zeros(4, **i32), torch.zeros(3, **i32))
    assert not w.any()


def test_offsets_past_32_bits(bsr):
    """The last pages of a pool of more than 2^32 bytes a tensor."""
    H, page, n = 2, 64, 150
    pages = (1 << 32) // (H * page * 256) + 40
    k, v, _, _ = bsr.paged_cache(pages, H, page)
    w = bsr.cache_weights(k)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, pages - 3, 5]], **i32)
    rs, kl = torch.tensor([0, n], **i32), torch.tensor([n], **i32)
    xk, xv = rows_of(n, H, seed=2)
    bsr.cache_write(xk, xv, k, v, table, rs, kl)
    q = torch.randn((n, 4, 128), device="cuda").bfloat16()
    for m in (1, n):
        r = torch.tensor([0, m], **i32)
        _, lse = bsr.paged_attn(q[:m], k, v, table, r, kl, max_new=m)
        bsr.cache_weigh(q[:m], lse, w, k, table, r, kl, max_new=m, accumulate=False)
        got = torch.cat([w[p] for p in table[0].tolist()], 1)[:, :n].double().cpu().numpy()
        ref, slack, count = OP.received(q[:m].double().cpu().numpy(), lse.double().cpu().numpy(), xk.double().cpu().numpy(),
                                        list(range(n - m, n)), n)
        assert np.all(np.abs(got - ref) <= 2 * 264 * U * slack + (2.0 ** -21 + (count + 8) * U) * ref + 1e-30)
    kept, _ = bsr.cache_evict(k, v, w, table, kl, 80, first=1, last=3)
    back = bsr.cache_read(k, v, table, torch.tensor([0, 80], **i32), torch.tensor([80], **i32), rows=80)
    for h in range(H):
        mine = kept[0, h].long()
        assert mine.tolist() == OP.survivors(got[h], 80, 1, 3)
        assert torch.equal(back[0][:, h], xk[mine, h]) and torch.equal(back[1][:, h], xv[mine, h])


# ---- what the device refuses

def test_bad_pages_are_reported_and_nothing_moves(bsr):
    for kind in ("bf16", "e4m3"):
        b, w = evict_case([200, 90], 2, 64, kind, seed=4)
        for bad in (-1, b.pages, 2 ** 31 - 1, -2 ** 31):
            t = b.table.clone()
            t[0, 3] = bad
            wt = torch.from_numpy(w).cuda()
            ws = torch.empty(256, dtype=torch.uint8, device="cuda")
            kept, new_len = bsr.cache_evict(b.k_pages, b.v_pages, wt, t, b.kv_len, 100, ws=ws, **b.exps)
            assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL
            assert (kept[0] == -1).all() and new_len.tolist() == [200, 90] and torch.equal(wt.cpu(), torch.from_numpy(w))
            to = torch.tensor([[0, bad], [1, 2]], dtype=torch.int32, device="cuda")
            bsr.cache_evict(b.k_pages, b.v_pages, wt.clone(), b.table, torch.tensor([200, 0], dtype=torch.int32, device="cuda"), 100,
                            to_table=to, ws=ws, **b.exps)
            assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL
            for news in (1, 60):
                q = torch.randn((news, 4, 128), device="cuda").bfloat16()
                lse = torch.zeros((news, 4), device="cuda")
                rs = torch.tensor([0, news, news], dtype=torch.int32, device="cuda")
                big = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
                bsr.cache_weigh(q, lse, wt, b.k_pages, t, rs, b.kv_len, max_new=news, k_exp=b.k_exp, ws=big)
                assert bsr.sparse_attn_last_device_status(big) == bsr.SA_EINVAL
                bsr.cache_weigh(q, lse, wt, b.k_pages, b.table, rs, b.kv_len, max_new=news, k_exp=b.k_exp, ws=big)
                assert bsr.sparse_attn_last_device_status(big) == 0


def test_bad_lengths_are_reported(bsr):
    b, w = evict_case([200, 90], 2, 64, "bf16", seed=4)
    wt = torch.from_numpy(w).cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for n in (-1, 100000):
        kl = torch.tensor([n, 90], dtype=torch.int32, device="cuda")
        before = [raw(b.k_pages), raw(b.v_pages)]
        kept, new_len = bsr.cache_evict(b.k_pages, b.v_pages, wt, b.table, kl, 100, ws=ws)
        assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL
        assert new_len.tolist() == [n, 90] and (kept[0] == -1).all() and (kept[1, :, :90] == torch.arange(90, device="cuda")).all()
        assert np.array_equal(raw(b.k_pages), before[0]) and np.array_equal(raw(b.v_pages), before[1])
    narrow = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")  # room for 64 of 90 tokens
    kept, _ = bsr.cache_evict(b.k_pages, b.v_pages, wt, b.table, torch.tensor([0, 90], dtype=torch.int32, device="cuda"), 100,
                              to_table=narrow, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL and (kept == -1).all()


def test_refusals_of_the_python_layer(bsr):
    b, w = evict_case([200, 90], 2, 64, "bf16", seed=4)
    wt = torch.from_numpy(w).cuda()
    call = lambda keep=50, w=wt, table=b.table, kl=b.kv_len, **kw: bsr.cache_evict(b.k_pages, b.v_pages, w, table, kl, keep, **kw)  # noqa: E731
    for bad in (dict(keep=0), dict(keep=-3), dict(first=-1), dict(last=-1), dict(first=30, last=21), dict(w=wt.double()),
                dict(w=wt[:1]), dict(w=wt.cpu()), dict(table=b.table.long()), dict(kl=b.kv_len.long()), dict(kl=b.kv_len[:1]),
                dict(to_table=b.table[:1]), dict(to_table=b.table[:, :0]), dict(to_table=b.table.long()), dict(k_exp=wt),
                dict(kept=torch.empty((2, 2, 49), dtype=torch.int32, device="cuda")), dict(new_len=torch.empty(3, dtype=torch.int32, device="cuda")),
                dict(ws=torch.empty(255, dtype=torch.uint8, device="cuda")), dict(keep=1 << 31)):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    with pytest.raises(bsr.SparseAttnError):
        call(new_len=b.kv_len)
    q = torch.randn((2, 4, 128), device="cuda").bfloat16()
    lse = torch.zeros((2, 4), device="cuda")
    rs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    weigh = lambda q=q, lse=lse, w=wt, **kw: bsr.cache_weigh(q, lse, w, b.k_pages, b.table, rs, b.kv_len, **kw)  # noqa: E731
    for bad in (dict(q=q[:, :3]), dict(q=q.half()), dict(lse=lse[:1]), dict(lse=lse.double()), dict(w=wt[:1]), dict(first=-1),
                dict(window=-1), dict(window=3, causal=False), dict(max_new=-1), dict(k_exp=wt),
                dict(ws=torch.empty(255, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            weigh(**bad)
    with pytest.raises(bsr.SparseAttnError):
        weigh(scale=0.0)


# ---- together

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_bounded_cache_in_use(bsr, kind):
    """Decoding under a budget: write, attend, weigh; evict when over it.
    Compared with a program that keeps every head's tokens in lists."""
    S, H, Hq, page, budget, slack, first, last = 2, 2, 4, 16, 48, 16, 2, 8
    per = (budget + slack) // page + 1
    k, v, ke, ve = bsr.paged_cache(S * per, H, page, kind)
    exps = dict(k_exp=ke, v_exp=ve)
    w = bsr.cache_weights(k)
    g = torch.Generator().manual_seed(0)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(S * per, generator=g).to(torch.int32).reshape(S, per).cuda()
    rs = torch.arange(S + 1, **i32)
    kl = torch.zeros(S, **i32)
    held = [[[] for _ in range(H)] for _ in range(S)]   # (k, v, weight) of each head's tokens
    for step in range(150):
        xk, xv = (torch.randn((S, H, 128), generator=g).bfloat16().cuda() for _ in range(2))
        q = (torch.randn((S, Hq, 128), generator=g) * 2).bfloat16().cuda()
        kl.add_(1)
        bsr.cache_write(xk, xv, k, v, table, rs, kl, **exps)
        o, lse = bsr.paged_attn(q, k, v, table, rs, kl, max_new=1, **exps)
        bsr.cache_weigh(q, lse, w, k, table, rs, kl, max_new=1, k_exp=ke)
        back = [t.double().cpu().numpy() for t in bsr.cache_read(k, v, table, rs, kl, rows=S, **exps)]
        q64, l64 = q.double().cpu().numpy(), lse.double().cpu().numpy()
        n = int(kl[0])
        for s in range(S):
            for h in range(H):
                held[s][h].append([back[0][s, h], back[1][s, h], 0.0])
                kk, vv = np.stack([t[0] for t in held[s][h]]), np.stack([t[1] for t in held[s][h]])
                heads = slice(2 * h, 2 * h + 2)
                ro, _, mass, reach = OP.paged_attention(q64[s:s + 1, heads], kk[:, None], vv[:, None], [n - 1], n)
                ds = 264 * U * reach
                tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (n + 64) * U)[..., None] * mass
                assert np.all(np.abs(o[s:s + 1, heads].double().cpu().numpy() - ro) <= tol), step
                got, _, _ = OP.received(q64[s:s + 1, heads], l64[s:s + 1, heads], kk[:, None], [n - 1], n)
                for t, x in zip(held[s][h], got[0]):
                    t[2] += x
        if n > budget + slack - 1:
            kept, new_len = bsr.cache_evict(k, v, w, table, kl, budget, first=first, last=last, **exps)
            kl.copy_(new_len)
            kept = kept.cpu().numpy()
            for s in range(S):
                for h in range(H):
                    ws = np.array([t[2] for t in held[s][h]])
                    mine = kept[s, h]
                    assert set(range(first)) <= set(mine) and set(range(n - last, n)) <= set(mine) and np.all(np.diff(mine) > 0)
                    gone = np.setdiff1d(np.arange(n), mine)
                    chosen = np.setdiff1d(mine, list(range(first)) + list(range(n - last, n)))
                    assert ws[gone].max() <= ws[chosen].min() * (1 + 1e-4)  # 150 steps of 2^-13 at most
                    held[s][h] = [held[s][h][j] for j in mine]
    assert int(kl[0]) < 150


# ---- waits, graphs, streams

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_wait_that_gives_up_is_reported(bsr, kind):
    from block_sparse_routed_gb300 import _native

    b = Batch([2900, 70], [300, 1], 2, 64, kind, seed=9)
    q, lse, w = run_weigh(bsr, b, 8, check=False)
    ws = bsr.weigh_workspace(q, b.k_pages, b.table, 300)
    call = lambda w: bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len, max_new=300, k_exp=b.k_exp, ws=ws)  # noqa: E731
    prev = _native.sparse_attn_set_single_probe_waits(True)
    try:
        statuses = []
        for _ in range(5):  # a single probe almost surely comes too early
            call(fresh_weights(b))
            statuses.append(bsr.sparse_attn_last_device_status(ws))
            if statuses[-1] == bsr.SA_ETIMEOUT:
                break
    finally:
        _native.sparse_attn_set_single_probe_waits(bool(prev))
    assert bsr.SA_ETIMEOUT in statuses
    w2 = fresh_weights(b)
    call(w2)
    assert bsr.sparse_attn_last_device_status(ws) == 0 and torch.equal(w, w2)


@pytest.mark.parametrize("news,keep", [(1, 100), (40, 5000)])
def test_captured(bsr, news, keep):
    """Attention, weights and eviction in one graph, replayed on new lengths."""
    b = Batch([9000, 300], [news, 1], 2, 64, "e4m3", seed=9)
    g = torch.Generator().manual_seed(1)
    q = torch.randn((b.rows, 8, 128), generator=g).bfloat16().cuda()
    start = [t.clone() for t in (b.k_pages.view(torch.uint8), b.v_pages.view(torch.uint8), b.k_exp, b.v_exp)] + [fresh_weights(b)]
    state = [t.clone() for t in start]
    o, lse = torch.zeros_like(q), torch.zeros((b.rows, 8), device="cuda")
    kept = torch.zeros((2, 2, keep), dtype=torch.int32, device="cuda")
    new_len = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws, ws2 = bsr.paged_workspace(q, b.k_pages, b.table, news), bsr.weigh_workspace(q, b.k_pages, b.table, news)

    def step():
        k, v = state[0].view(torch.float8_e4m3fn), state[1].view(torch.float8_e4m3fn)
        bsr.paged_attn(q, k, v, b.table, b.row_start, b.kv_len, max_new=news, k_exp=state[2], v_exp=state[3], o=o, lse=lse, ws=ws)
        bsr.cache_weigh(q, lse, state[4], k, b.table, b.row_start, b.kv_len, max_new=news, k_exp=state[2], ws=ws2)
        bsr.cache_evict(k, v, state[4], b.table, b.kv_len, keep, first=2, last=50, k_exp=state[2], v_exp=state[3], kept=kept, new_len=new_len)

    def reset():
        for t, x in zip(state, start):
            t.copy_(x)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([9000, 300], [4999, 123]):
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        reset()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (*state, o, lse, kept, new_len)]
        for _ in range(2):
            reset()
            kept.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(want, (*state, o, lse, kept, new_len)))
        assert new_len.tolist() == [min(n, keep) for n in lens]


def test_two_streams_at_once(bsr):
    """Calls on two streams, each with workspaces of its own, give what they give alone."""
    cases = []
    for seed, news in ((1, 300), (2, 200)):
        b = Batch([4000, 200], [news, 1], 4, 64, "bf16", seed=seed)
        q = torch.randn((b.rows, 8, 128), device="cuda").bfloat16()
        _, lse = bsr.paged_attn(q, *b.where)
        w = fresh_weights(b)
        bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len)
        cases.append((b, q, lse, w))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        out = []
        for s, (b, q, lse, _) in zip(streams, cases):
            with torch.cuda.stream(s):
                w = fresh_weights(b)
                bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len)
                k, v = b.k_pages.clone(), b.v_pages.clone()
                kept, _ = bsr.cache_evict(k, v, w.clone(), b.table, b.kv_len, 1000, first=4, last=4)
                out.append((w, kept))
        torch.cuda.synchronize()
        for (w, kept), (b, _, _, want) in zip(out, cases):
            assert torch.equal(w, want)
            j = np.arange(4000)
            for h in range(4):
                assert kept[0, h].tolist() == OP.survivors(want.cpu().numpy()[b.table_np[0, j // 64], h, j % 64], 1000, 4, 4)


@pytest.mark.parametrize("H,Hq,news", [(1, 1, 1200), (1, 100, 30), (2, 192, 5), (1, 97, 40), (7, 49, 90)])
def test_weights_of_odd_groups(bsr, H, Hq, news):
    """Groups that leave rows of a step unused, and groups wider than a step."""
    b = Batch([1300, 50], [news, 3], H, 32, "bf16", seed=21)
    run_weigh(bsr, b, Hq)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [16, 17, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("H,group,causal,window", [(2, 1, True, 0), (1, 1, False, 0), (3, 1, True, 90)])
def test_weights_by_rows(bsr, kind, news, H, group, causal, window):
    """Around the numbers of rows at which the form changes; beside them sequences of other numbers."""
    b = Batch([400, 700, 33, 140], [news, 1, 9, news // 2], H, 64, kind, seed=news, first_row=1, after=1)
    run_weigh(bsr, b, H * group, causal=causal, window=window, accumulate=news % 2 == 0)


@pytest.mark.parametrize("news", [1, 3, 11, 37, 64, 80])
def test_an_infinite_key_that_all_rows_reject(bsr, news):
    """Each row's logit is -inf there: it weighs nothing, whatever stands beside the rows."""
    b = Batch([300, 90], [news, 1], 2, 64, seed=4)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    q[:, :, 5] = -q[:, :, 5].abs() - 1
    pg, sl = b.table_np[0, 2], 7  # token 135
    b.k_pages[pg, 1, sl] = 0.5
    b.k_pages[pg, 1, sl, 5] = math.inf
    _, lse = bsr.paged_attn(q, *b.where)
    assert lse.isfinite().all()
    w = bsr.cache_weights(b.k_pages)
    bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len, accumulate=False)
    assert w.isfinite().all() and w[pg, 1, sl] == 0 and w[pg, 0, sl] > 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 20, 200])
def test_weights_without_a_workspace(bsr, kind, news):
    """The status goes unreported, and a bad sequence is left as it was all the same."""
    b = Batch([300, 90, 50], [news, 1, 1], 2, 64, kind, seed=4)
    q, lse, want = run_weigh(bsr, b, 4)
    w = fresh_weights(b)
    bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len, max_new=news, k_exp=b.k_exp)
    assert torch.equal(w, want)
    kl = b.kv_len.clone()
    kl[1] = b.table.shape[1] * 64 + 1
    w = fresh_weights(b)
    bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, kl, max_new=news, k_exp=b.k_exp)
    pages = b.table_np[1, :2]
    assert torch.equal(w[pages], fresh_weights(b)[pages])
    for s in (0, 2):
        pages = b.table_np[s, : (b.lens[s] + 63) // 64]
        assert torch.equal(w[pages], want[pages])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H", [2, 40])  # eight blocks a unit, and two
@pytest.mark.parametrize("shape", ["rising", "falling", "hill", "valley", "steps", "late gap"])
def test_eviction_in_place_of_uneven_gaps(bsr, kind, H, shape):
    """Tokens that go stand together: places catch up with sources of other
    rounds, or never do."""
    n, keep = (9505, 5000) if H == 2 else (3000, 1700)
    b, w = evict_case([n], H, 64, kind, seed=11)
    x = np.arange(n) / n
    level = {"rising": x, "falling": -x, "hill": -np.abs(x - 0.6), "valley": np.abs(x - 0.3), "steps": np.floor(x * 40) % 2,
             "late gap": -(np.abs(x - 0.7) < 0.25).astype(float)}[shape]
    j = np.arange(n)
    for h in range(H):
        w[b.table_np[0, j // 64], h, j % 64] = (level * (1 + h % 3) + 1e-3 * w[b.table_np[0, j // 64], h, j % 64]).astype(np.float32)
    run_evict(bsr, b, w, keep, 4, 50)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,group", [(64, 1), (65, 1), (96, 1), (100, 1), (128, 1), (81, 1), (16, 7), (40, 2), (41, 2)])
def test_weights_of_as_many_rows_each(bsr, kind, news, group):
    """Where the mean number of rows decides on the form."""
    b = Batch([400, 333, news], [news] * 3, 2, 64, kind, seed=news, first_row=1, after=1)
    run_weigh(bsr, b, 2 * group, accumulate=news % 2 == 0)


def test_a_workspace_follows_the_rows(bsr):
    table = torch.zeros((8, 4), dtype=torch.int32, device="cuda")
    k = bsr.paged_cache(16, 2, 64)[0]
    size = lambda rows, max_new: bsr.weigh_workspace(torch.zeros((rows, 2, 128), dtype=torch.bfloat16, device="cuda"), k, table, max_new).numel()  # noqa: E731
    assert size(8 * 64, 64) == size(8 * 80, 128) == 256
    assert size(8 * 80 + 8, 128) > 256 and size(200, 200) > 256
