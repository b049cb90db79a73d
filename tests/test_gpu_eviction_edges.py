"""Weights and eviction at their edges: values that are not numbers, rows that
count nothing, tables wider than their sequences."""

import math

import numpy as np
import pytest

from oracle import paged as OP

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from .test_gpu_eviction import check_weights, evict_case, fresh_weights, run_evict  # noqa: E402
from .test_gpu_paged import U, Batch, bsr  # noqa: E402,F401

FORMS = {"few": 3, "mid": 30, "chunk": 200}  # rows of the first sequence, 4 / 2 heads


def form_batch(bsr, form, kind, seed=4):
    """A batch that the form takes, its Q, lse and maximal number of rows."""
    news = FORMS[form]
    b = Batch([300, 90], [news, 1], 2, 64, kind, seed=seed)
    q = torch.randn((b.rows, 4, 128), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    assert (bsr.weigh_workspace(q, b.k_pages, b.table, news).numel() > 256) == (form == "chunk")
    _, lse = bsr.paged_attn(q, *b.where, max_new=news, **b.exps)
    return b, q, lse, news


def weigh(bsr, b, q, lse, news, w=None, k=None, ke=None, **kw):
    w = fresh_weights(b) if w is None else w
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    bsr.cache_weigh(q, lse, w, b.k_pages if k is None else k, b.table, b.row_start, b.kv_len, max_new=news,
                    k_exp=b.k_exp if ke is None else ke, ws=ws, **kw)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    return w


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", FORMS)
def test_rows_without_a_sum_in_every_form(bsr, kind, form):
    """lse = -inf (a row that saw no key) and +inf."""
    b, q, lse, news = form_batch(bsr, form, kind)
    lse[0, 1], lse[b.rows - 1, 3] = -math.inf, math.inf
    before = fresh_weights(b).cpu().numpy()
    w = weigh(bsr, b, q, lse, news)
    lse[lse == math.inf] = -math.inf  # to the oracle: no such row
    check_weights(b, q, lse, before, w, 0, True)


def spoil(b, s, j, h, value):
    """Copies of K and its exponents with one key that is not a number, or infinite."""
    k, ke = b.k_pages.clone(), None if b.k_exp is None else b.k_exp.clone()
    pg, sl = b.table_np[s, j // b.page], j % b.page
    if ke is None:
        k[pg, h, sl, 5] = value
    else:
        ke[pg, h, sl] = 255
    return k, ke, (pg, h, sl)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("j", [0, 135, 299])
def test_a_key_that_is_nan_in_every_form(bsr, kind, form, j):
    b, q, lse, news = form_batch(bsr, form, kind)
    clean = weigh(bsr, b, q, lse, news)
    k, ke, at = spoil(b, 0, j, 1, math.nan)
    w = weigh(bsr, b, q, lse, news, k=k, ke=ke)
    assert w[at].isnan()
    w[at] = clean[at]
    assert torch.equal(w, clean)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", FORMS)
def test_rows_that_count_nothing_may_hold_anything(bsr, kind, form):
    b, q, lse, news = form_batch(bsr, form, kind)
    for r, h, value in ((0, 1, math.nan), (news // 2, 2, math.inf), (news - 1, 0, -math.inf), (news, 3, math.nan)):
        q[r, h] = value
        lse[r, h] = -math.inf
    before = fresh_weights(b).cpu().numpy()
    w = weigh(bsr, b, q, lse, news)
    check_weights(b, q, lse, before, w, 0, True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("causal", [True, False])
def test_a_key_that_no_counting_row_sees(bsr, kind, form, value, causal):
    """The last token, seen by the last row alone, whose lse says that it counts nothing."""
    b, q, lse, news = form_batch(bsr, form, kind)
    if causal:
        lse[news - 1] = -math.inf
    else:
        lse[:news] = -math.inf
    clean = weigh(bsr, b, q, lse, news, causal=causal)
    k, ke, at = spoil(b, 0, 299, 1, value)
    w = weigh(bsr, b, q, lse, news, k=k, ke=ke, causal=causal)
    assert w[at] == 0 and torch.equal(w, clean)


def microseconds(call):
    best = math.inf
    for _ in range(5):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        call()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) * 1e3)
    return best


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("what", ["lse", "row", "key"])
def test_one_nan_in_a_chunk(bsr, kind, what):
    """It reaches the keys that the row sees, or the rows that see the key, no
    other sequence, and does not make the call longer by orders of magnitude."""
    b = Batch([2900, 700], [300, 250], 2, 64, kind, seed=9)
    q = torch.randn((b.rows, 8, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    _, lse = bsr.paged_attn(q, *b.where, max_new=300, **b.exps)
    clean = weigh(bsr, b, q, lse, 300)
    k, ke = b.k_pages, b.k_exp
    if what == "lse":
        lse2, q2 = lse.clone(), q
        lse2[280, 5] = math.nan  # key head 1
    else:
        q2 = q.clone()
        if what == "row":
            q2[280, 5, 77] = math.nan
        else:
            k, ke, _ = spoil(b, 0, 3, 1, math.nan)
        _, lse2 = bsr.paged_attn(q2, k, *b.where[1:], max_new=300, k_exp=ke, v_exp=b.v_exp)
    w = weigh(bsr, b, q2, lse2, 300, k=k, ke=ke)
    seen = 2900 - 300 + 281 if what != "key" else 2900
    bad = torch.zeros_like(w, dtype=torch.bool)
    for j in range(seen):
        bad[b.table_np[0, j // 64], 1, j % 64] = True
    assert w[bad].isnan().all() and torch.equal(w[~bad], clean[~bad])
    ws = bsr.weigh_workspace(q, b.k_pages, b.table, 300)
    scratch = clean.clone()
    call = lambda l, x, k, ke: bsr.cache_weigh(x, l, scratch, k, b.table, b.row_start, b.kv_len, max_new=300, k_exp=ke, ws=ws)  # noqa: E731
    fine = microseconds(lambda: call(lse, q, b.k_pages, b.k_exp))
    odd = microseconds(lambda: call(lse2, q2, k, ke))
    assert odd < 20 * fine, (odd, fine)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_pages_are_reported_by_the_form_for_chunks(bsr, kind):
    b = Batch([300, 290], [200, 200], 2, 64, kind, seed=4)
    q = torch.randn((b.rows, 4, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    _, lse = bsr.paged_attn(q, *b.where, max_new=200, **b.exps)
    clean = weigh(bsr, b, q, lse, 200)
    ws = bsr.weigh_workspace(q, b.k_pages, b.table, 200)
    assert ws.numel() > 256
    for bad in (-1, b.pages, 2 ** 31 - 1, -2 ** 31):
        t = b.table.clone()
        t[0, 3] = bad
        w = fresh_weights(b)
        bsr.cache_weigh(q, lse, w, b.k_pages, t, b.row_start, b.kv_len, max_new=200, k_exp=b.k_exp, ws=ws)
        assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL
        lost = int(b.table_np[0, 3])
        assert torch.equal(w[lost], fresh_weights(b)[lost])  # (nobody's row names it)
        w[lost] = clean[lost]
        assert torch.equal(w, clean)
        bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len, max_new=200, k_exp=b.k_exp, ws=ws)
        assert bsr.sparse_attn_last_device_status(ws) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("to", [False, True])
@pytest.mark.parametrize("lens,H,keep", [([1100, 300], 2, 700), ([700, 40, 333], 60, 200)])  # eight blocks a unit, and one
def test_eviction_under_a_wide_table(bsr, kind, to, lens, H, keep):
    """Entries past a sequence's pages are not looked at, however many there are."""
    b, w = evict_case(lens, H, 64, kind, seed=3)
    wide = torch.full((len(lens), 4096), -7, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    run_evict(bsr, b, w, keep, 4, 50, to)


def check_scaled(bsr, kind, news, qe, ke, se):
    """Q near 2^qe (zeros below BF16's range), K near 2^ke, scale 2^se, lse by the oracle."""
    n, scale = 333, 2.0 ** se
    g = torch.Generator().manual_seed(2)
    b = Batch([n], [news], 1, 64, kind, seed=3)
    x = (torch.randn((n, 1, 128), generator=g) * 2.0 ** ke).bfloat16().cuda()
    rs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    bsr.cache_write(x, x, b.k_pages, b.v_pages, b.table, rs, b.kv_len, **b.exps)
    k = bsr.cache_read(b.k_pages, b.v_pages, b.table, rs, b.kv_len, rows=n, **b.exps)[0].double().cpu().numpy()
    q = ((0.25 + torch.rand((news, 4, 128), generator=g)) * 2.0 ** qe).bfloat16().cuda()
    pos = list(range(n - news, n))
    lse = torch.from_numpy(OP.paged_attention(q.double().cpu().numpy(), k, k, pos, n, scale=scale)[1]).float().cuda()
    w = bsr.cache_weights(b.k_pages)
    bsr.cache_weigh(q, lse, w, b.k_pages, b.table, b.row_start, b.kv_len, max_new=news, k_exp=b.k_exp, scale=scale)
    got = torch.cat([w[p] for p in b.table[0].tolist()[:6]], 1)[:, :n].double().cpu().numpy()
    ref, slack, count = OP.received(q.double().cpu().numpy(), lse.double().cpu().numpy(), k, pos, n, scale=scale)
    assert np.all(np.abs(got - ref) <= 2 * 264 * U * slack + (2.0 ** -21 + (count + 8) * U) * ref + count * 2.0 ** -126)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 4, 20, 300])  # the two kernels for few rows, the one for more, chunks
@pytest.mark.parametrize("qe,ke,se", [(120, -117, -5), (-117, 120, -5), (60, -58, -4), (50, 50, -100), (0, 100, -100), (100, 0, -100),
                                      (-62, 0, 60), (0, -62, 60), (60, -120, 58)])
def test_logits_of_large_and_small_factors(bsr, kind, news, qe, ke, se):
    check_scaled(bsr, kind, news, qe, ke, se)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 4, 20, 300])
@pytest.mark.parametrize("ke,se", [(0, 0), (119, 60), (119, -100), (-117, 60), (-117, -100)])
def test_rows_of_zeros_weigh_all_keys_alike(bsr, kind, news, ke, se):
    check_scaled(bsr, kind, news, -200, ke, se)


@pytest.mark.parametrize("to", [False, True])
def test_pages_that_must_not_be_shared(bsr, to):
    """Two sequences of one table's row over their budget, longer than the weights
    that shared memory holds: what stays is anyone's guess, but all of it are
    positions, and nothing lies outside of the call's tensors."""
    H, page, n, keep = 80, 128, 50001, 20000
    need, more = -(-n // page), -(-keep // page)
    pages = need + 2 * more + 1
    k, v, ke, ve = bsr.paged_cache(pages, H, page, "e4m3")
    for t in (k, v):
        t.view(torch.uint8).fill_(8)
    ke.fill_(120), ve.fill_(121)
    w = torch.rand((pages, H, page), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    table = torch.arange(need, dtype=torch.int32, device="cuda").repeat(2, 1)
    to_table = need + torch.arange(2 * more, dtype=torch.int32, device="cuda").reshape(2, more)
    kl = torch.full((2,), n, dtype=torch.int32, device="cuda")
    pool = torch.full((2 * H * keep + 2048,), -5, dtype=torch.int32, device="cuda")
    kept = pool[1024:-1024].view(2, H, keep)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    spare = w[-1].clone()
    _, new_len = bsr.cache_evict(k, v, w, table, kl, keep, first=3, last=70, to_table=to_table if to else None, k_exp=ke, v_exp=ve,
                                 kept=kept, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == 0 and new_len.tolist() == [keep] * 2
    assert int(kept.min()) >= 0 and int(kept.max()) < n
    assert (pool[:1024] == -5).all() and (pool[-1024:] == -5).all() and torch.equal(w[-1], spare)
    assert (kept[:, :, :3] == torch.arange(3, device="cuda")).all() and (kept[:, :, -70:] == torch.arange(n - 70, n, device="cuda")).all()
