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


# ---- values that are not finite

def check_odd(b, q, o, lse, causal=True, window=0):
    """Every row as the float64 oracle has it: NaN and infinities where it has
    them, what is finite within the bounds."""
    og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
    q64 = q.double().cpu().numpy()
    finite = []
    for s, n in enumerate(b.lens):
        if not b.news[s]:
            continue
        rows, pos = (list(x) for x in zip(*OP.positions(b.starts, b.lens, s)))
        k, v = OP.gather(b.k64, b.table_np, s, n), OP.gather(b.v64, b.table_np, s, n)
        with np.errstate(invalid="ignore", over="ignore"):
            ro, rl, mass, reach = OP.paged_attention(q64[rows], k, v, pos, n, causal, window)
            fine = np.isfinite(ro)
            assert np.array_equal(np.isnan(ro), np.isnan(og[rows])), s
            assert np.array_equal(ro[np.isinf(ro)], og[rows][np.isinf(ro)]), s
            ds = (2 * 128 + 8) * U * np.where(np.isfinite(reach), reach, 0)
            tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (n + 64) * U)[..., None] * mass
            assert np.all(np.abs(og[rows] - ro)[fine] <= tol[fine]), s
            assert np.array_equal(np.isnan(rl), np.isnan(lg[rows])), s
            assert np.array_equal(rl == -np.inf, lg[rows] == -np.inf), s
            tl = ds + 2 * (n + 64) * U + 2.0 ** -21 + 4 * U * np.abs(rl)
            known = np.isfinite(rl)
            assert np.all(np.abs(lg[rows] - rl)[known] <= tl[known]), s
        finite.append(fine.reshape(-1))
    finite = np.concatenate(finite)
    return finite


def set_nan(b, what, s, j):
    """Key or value of token j of sequence s is NaN (BF16: one dimension of it)."""
    pg, sl = b.table_np[s, j // b.page], j % b.page
    t, t64, e = (b.k_pages, b.k64, b.k_exp) if what == "k" else (b.v_pages, b.v64, b.v_exp)
    if b.kind == "e4m3":
        e[pg, :, sl] = 255
        t64[pg, :, sl] = math.nan
    else:
        t[pg, :, sl, 17] = math.nan
        t64[pg, :, sl, 17] = math.nan


@KINDS
@pytest.mark.parametrize("lens,news,H,Hq,window", [
    ([65, 17, 161], [1, 1, 1], 2, 8, 0),         # the newest key is alone in its sixteen
    ([161, 33], [4, 3], 1, 4, 0),                # 12 to 16 packed rows
    ([3000, 81], [1, 1], 1, 4, 16),              # it is alone in the window's last sixteen
    ([81, 161], [70, 90], 1, 2, 0),              # chunks: alone in its key tile
    ([500, 161], [60, 1], 1, 4, 1),              # every row sees one key
])
def test_a_nan_key_alone_among_the_keys_of_a_warp(bsr, kind, lens, news, H, Hq, window):
    b = Batch(lens, news, H, 64, kind, seed=3)
    for s, n in enumerate(lens):
        set_nan(b, "k", s, n - 1)
    q, o, lse = run_attention(bsr, b, Hq, window=window)
    check_odd(b, q, o, lse, True, window)
    assert lse.isnan().any()


def run_with(bsr, b, q, **kw):
    ws = bsr.paged_workspace(q, b.k_pages, b.table, max(b.news))
    o, lse = bsr.paged_attn(q, *b.where, max_new=max(b.news), **b.exps, ws=ws, **kw)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    return o, lse


@KINDS
@pytest.mark.parametrize("lens,news,H,Hq", [
    ([40, 5], [1, 1], 1, 4),                     # one part
    ([9505, 100], [1, 1], 2, 8),                 # cut into many and joined
    ([9505, 100], [4, 2], 1, 4),
    ([100, 70], [60, 30], 1, 2),
    ([9505, 100], [150, 40], 1, 4),
])
def test_a_nan_in_a_query_row(bsr, kind, lens, news, H, Hq):
    """One head of one row has a NaN: its output and its log-sum-exp are NaN
    (-inf would say that it sees no key), and no other's."""
    b = Batch(lens, news, H, 64, kind, seed=3)
    q = (torch.randn((b.rows, Hq, 128), generator=torch.Generator().manual_seed(5)).bfloat16() * 2).cuda()
    q[0, 1, 77] = math.nan
    o, lse = run_with(bsr, b, q)
    check_odd(b, q, o, lse)
    assert lse.isnan().sum() == 1 and o.isnan().sum() == 128


@KINDS
@pytest.mark.parametrize("news", [1, 3, 40])
def test_a_nan_value_whose_probability_vanishes(bsr, kind, news):
    """0 * NaN is NaN: a NaN that a row sees is not lost where its key's
    probability is below every number of 32 bits."""
    n = 200
    b = Batch([n], [news], 1, 64, kind, seed=3)
    q = torch.ones((news, 4, 128), dtype=torch.bfloat16, device="cuda")
    # token 0: logit -40 * sqrt(128) = -452, the others' near 0
    pg = b.table_np[0, 0]
    if kind == "bf16":
        b.k_pages[pg, 0, 0] = -40.0
    else:
        b.k_pages.view(torch.uint8)[pg, 0, 0] = 0xF8  # -256
        b.k_exp[pg, 0, 0] = 127 - 2
    b.k64[pg, 0, 0] = -40.0 if kind == "bf16" else -64.0
    set_nan(b, "v", 0, 0)
    o, lse = run_with(bsr, b, q)
    if kind == "bf16":
        assert o[:, :, 17].isnan().all() and o.isnan().sum() == news * 4
    else:
        assert o.isnan().all()
    assert lse.isfinite().all()


# ---- the ends of the formats' ranges

class Filled:
    """One sequence in a cache that cache_write has filled with the rows k, v
    [n, H, 128]; k64, v64 are what it then holds."""

    def __init__(self, bsr, k, v, news, page=64, kind="bf16"):
        n, H, _ = k.shape
        i32 = dict(dtype=torch.int32, device="cuda")
        pages = -(-n // page)
        self.cache = bsr.paged_cache(pages, H, page, kind)
        self.exps = dict(k_exp=self.cache[2], v_exp=self.cache[3])
        self.table = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).to(torch.int32)[None].cuda()
        self.kv_len, self.n, self.news = torch.tensor([n], **i32), n, news
        self.row_start = torch.tensor([0, news], **i32)
        all_rows = torch.tensor([0, n], **i32)
        bsr.cache_write(k.bfloat16().cuda(), v.bfloat16().cuda(), *self.cache[:2], self.table, all_rows, self.kv_len,
                        **self.exps)
        back = bsr.cache_read(*self.cache[:2], self.table, all_rows, self.kv_len, rows=n, **self.exps)
        self.k64, self.v64 = (t.double().cpu().numpy() for t in back)

    def attend(self, bsr, q, **kw):
        return bsr.paged_attn(q, *self.cache[:2], self.table, self.row_start, self.kv_len, **self.exps, **kw)

    def check(self, q, o, lse, **kw):
        ro, rl, mass, reach = OP.paged_attention(q.double().cpu().numpy(), self.k64, self.v64,
                                                 list(range(self.n - self.news, self.n)), self.n, **kw)
        assert np.isfinite(ro).all()
        ds = (2 * 128 + 8) * U * reach
        tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (self.n + 64) * U)[..., None] * mass
        assert np.all(np.abs(o.double().cpu().numpy() - ro) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - rl) <= ds + 2 * (self.n + 64) * U + 2.0 ** -21 + 4 * U * np.abs(rl))


@KINDS
@pytest.mark.parametrize("news", [1, 4, 40, 300])
@pytest.mark.parametrize("slope", [0.004, 0.02])
def test_large_values_under_rising_logits(bsr, kind, news, slope):
    """Values near 2^122 and logits that rise from key to key by 0.065 or 0.33
    (base 2): at the end of the walk sum 2^(x_j - max) is at most 23, so that
    sum 2^(x_j - max) |v_j| stays under 2^127, and the result must be finite
    however far the running reference lags."""
    n, H = 1500, 64 if news < 16 else 1  # (64 heads: a block walks several key tiles)
    k = (slope * torch.arange(n, dtype=torch.float32))[:, None, None].expand(n, H, 128)
    g = torch.Generator().manual_seed(1)
    v = (0.5 + 0.5 * torch.rand((n, 1, 128), generator=g)).expand(n, H, 128) * 2.0 ** 122
    f = Filled(bsr, k, v, news, kind=kind)
    q = torch.ones((news, 4 * H, 128), dtype=torch.bfloat16, device="cuda")
    f.check(q, *f.attend(bsr, q))


@KINDS
@pytest.mark.parametrize("news", [1, 4, 40])
@pytest.mark.parametrize("qe,ke", [(120, -117), (-117, 120), (60, -58), (0, 0)])
def test_logits_of_large_queries_and_small_keys(bsr, kind, news, qe, ke):
    """Q near 2^120 and K near 2^-117 and the reverse: their products are
    ordinary numbers, whatever the order in which scales are applied."""
    n = 333
    g = torch.Generator().manual_seed(2)
    k = torch.randn((n, 1, 128), generator=g) * 2.0 ** ke
    v = torch.randn((n, 1, 128), generator=g)
    f = Filled(bsr, k, v, news, kind=kind)
    q = ((0.25 + torch.rand((news, 4, 128), generator=g)) * 2.0 ** (qe - 2)).bfloat16().cuda()
    f.check(q, *f.attend(bsr, q))


@pytest.mark.parametrize("H", [1, 3, 8])
def test_the_largest_values_stay_finite(bsr, H):
    """256 * 2^120 is no BF16 number: what would round to it takes 240 * 2^120,
    which is at most half a step (2^-4) off."""
    n = 20
    x = torch.randn((n, H, 128), generator=torch.Generator().manual_seed(3))
    top = [3.3895e38, 3.31e38, 248 * 2.0 ** 120, 247 * 2.0 ** 120, 3.2e38, 2.0 ** 127, 2.0 ** 120]
    for i, t in enumerate(top):
        x[i, i % H] *= t / 4
        x[i, i % H, 5:9] = torch.tensor([t, -t, t / 2, -t / 3])
    x[8, 0, 3], x[8, 0, 4] = math.inf, 3.3895e38
    x[9, 0, 3], x[9, 0, 4] = math.nan, 3.3895e38
    x = x.clamp(-3.3895e38, 3.3895e38).where(x.isfinite(), x).bfloat16()
    b = Batch([n], [n], H, 16, "e4m3")
    xc = x.cuda()
    bsr.cache_write(xc, xc, *b.where, **b.exps)
    for j in range(n):
        pg, sl = b.table_np[0, j // 16], j % 16
        for h in range(H):
            want, byte = OP.quantise_row(bits(x[j, h]))
            for t, e in ((b.k_pages, b.k_exp), (b.v_pages, b.v_exp)):
                code = t.view(torch.uint8)[pg, h, sl].cpu().numpy()
                assert e[pg, h, sl].item() == byte
                assert np.all((code == want) | ((code & 127 == 127) & (want & 127 == 127))), (j, h)
    k, _ = bsr.cache_read(*b.where, rows=n, **b.exps)
    k, x = k.double().cpu(), x.double()
    fine = x.isfinite().all(-1)
    assert k[fine].isfinite().all() and k[~fine].isnan().all()
    err, amax = (k - x).abs()[fine], x.abs().amax(-1, keepdim=True).expand_as(x)[fine]
    # half a step, or half of the smallest step of a row whose largest code is 240 or more
    assert (err <= torch.maximum(2.0 ** -4 * x.abs()[fine], 2.0 ** -10 * amax / 224)).all()


@KINDS
@pytest.mark.parametrize("news", [1, 4, 40, 300])
def test_the_largest_values_reach_only_the_rows_that_see_them(bsr, kind, news):
    """Values of 3.39e38 in the newest tokens: rows that do not see them have
    the results of a cache without, the others finite ones."""
    n = 400
    g = torch.Generator().manual_seed(4)
    k, v = torch.randn((n, 1, 128), generator=g), torch.randn((n, 1, 128), generator=g)
    for j in (n - 1, n - 1 - news // 2):
        v[j, 0, 10:20] = 3.3895e38
        v[j, 0, 20:30] = -3.3895e38
    f = Filled(bsr, k, v, news, kind=kind)
    q = torch.randn((news, 4, 128), generator=g).bfloat16().cuda()
    f.check(q, *f.attend(bsr, q))


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("news", [1, 3, 40])
def test_nan_codes_under_a_finite_exponent(bsr, what, news):
    """A foreign code 127 in the newest token: NaN or 480 times its scale to
    the rows that see it, nothing to the others, in either form."""
    n = 100
    b = Batch([n, 70], [news, 1], 1, 64, "e4m3", seed=3)
    q = torch.randn((b.rows, 4, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    base, _ = run_with(bsr, b, q)
    pages, p64, exp = (b.k_pages, b.k64, b.k_exp) if what == "k" else (b.v_pages, b.v64, b.v_exp)
    pg, sl = b.table_np[0, (n - 1) // 64], (n - 1) % 64
    pages.view(torch.uint8)[pg, 0, sl, 9] = 127
    exp[pg, 0, sl] = 127
    p64[pg, 0, sl] = OP.dequantise(pages.view(torch.uint8)[pg, 0, sl].cpu().numpy()[None], np.array([127]))[0]
    p64[pg, 0, sl, 9] = 480.0
    o, _ = run_with(bsr, b, q)
    last = np.array([news - 1])
    others = np.setdiff1d(np.arange(b.rows), last)
    assert torch.equal(o[others], base[others])
    k, v = OP.gather(b.k64, b.table_np, 0, n), OP.gather(b.v64, b.table_np, 0, n)
    ro, _, mass, reach = OP.paged_attention(q.double().cpu().numpy()[last], k, v, [n - 1], n)
    got = o.double().cpu().numpy()[last]
    ds = (2 * 128 + 8) * U * reach
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (n + 64) * U)[..., None] * mass
    assert np.all(np.isnan(got) | (np.abs(got - ro) <= tol))


# ---- arguments and streams

@pytest.mark.parametrize("news", [1, 40])
def test_a_window_past_32_bits_is_all_keys(bsr, news):
    b = Batch([300, 70], [news, 1], 1, 64, seed=3)
    q = torch.randn((b.rows, 4, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want, lse = run_with(bsr, b, q)
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 + 1, 10 ** 30):
        o, l2 = run_with(bsr, b, q, window=window)
        assert torch.equal(o, want) and torch.equal(l2, lse), window


def test_tensors_of_another_shape_are_refused(bsr):
    b = Batch([200, 90], [4, 1], 2, 64, "e4m3", seed=4)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q = torch.randn((b.rows, 4, 128), **bf)
    for o in (torch.empty((4, b.rows, 128), **bf), torch.empty(b.rows * 512, **bf), torch.empty((b.rows, 512), **bf)):
        with pytest.raises(ValueError, match="o:"):
            bsr.paged_attn(q, *b.where, **b.exps, o=o)
    for lse in (torch.empty((4, b.rows), device="cuda"), torch.empty(4 * b.rows, device="cuda")):
        with pytest.raises(ValueError, match="lse"):
            bsr.paged_attn(q, *b.where, **b.exps, lse=lse)
    for name in ("k", "v"):
        with pytest.raises(ValueError, match=name):
            bsr.cache_read(*b.where, **b.exps, rows=b.rows, **{name: torch.empty((2, b.rows, 128), **bf)})
    for name in ("k_exp", "v_exp"):
        exps = dict(b.exps, **{name: b.exps[name].reshape(2, -1, 64)})
        with pytest.raises(ValueError, match=name):
            bsr.paged_attn(q, *b.where, **exps)
    # rows, outputs and a leading 1
    o, lse = bsr.paged_attn(q, *b.where, **b.exps)
    o1, l1 = bsr.paged_attn(q[None], *b.where, **b.exps, o=torch.empty((1, b.rows, 4, 128), **bf),
                            lse=torch.empty((1, b.rows, 4), device="cuda"))
    assert torch.equal(o1[0], o) and torch.equal(l1[0], lse)
    k, v = bsr.cache_read(*b.where, **b.exps, rows=b.rows)
    k1, _ = bsr.cache_read(*b.where, **b.exps, k=torch.empty((1, b.rows, 2, 128), **bf), v=torch.empty_like(v))
    assert torch.equal(k1[0], k)


def written_late(sizes):
    """Tensors of the current stream's pool that are given back at once, with
    writes to them that come late."""
    ts = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for t in ts:
        t.fill_(7)


@pytest.mark.parametrize("call", ["attn", "read"])
def test_what_a_call_on_another_stream_allocates_is_that_streams(bsr, call):
    """Memory that the current stream has freed may still be written there: a
    call on another stream, whose inputs alone are ready, must not get it."""
    b = Batch([300, 70], [40, 1], 2, 64, seed=9)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    side = torch.cuda.Stream()

    def run(**kw):
        if call == "attn":
            return bsr.paged_attn(q, *b.where, **kw)
        return bsr.cache_read(*b.where, rows=b.rows, **kw)

    want = run()
    sizes = [(t.shape, t.dtype) for t in want]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    if call == "attn":
        sizes.append(((bsr.paged_ws_bytes(q, b.k_pages, b.table),), torch.uint8))
    written_late(sizes)
    got = run(stream=side)
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("call", ["attn", "read"])
def test_outputs_of_a_call_on_another_stream_may_be_used_here(bsr, call):
    """They are used on the current stream, which waits for the other, and
    dropped: the next call on the other stream must not get their memory while
    that use is under way."""
    b = Batch([300, 70], [40, 1], 2, 64, seed=9)
    q1, q2 = (torch.randn((b.rows, 4, 128), device="cuda").bfloat16() for _ in range(2))
    k2 = torch.roll(b.k_pages, 1, 0).contiguous()
    side = torch.cuda.Stream()

    def run(i, **kw):
        if call == "attn":
            return bsr.paged_attn((q1, q2)[i], *b.where, **kw)
        return bsr.cache_read((b.k_pages, k2)[i], *b.where[1:], rows=b.rows, **kw)

    want = run(0)[0].clone()
    torch.cuda.synchronize()
    out = run(0, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    kept = out.clone()
    del out
    run(1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_a_stream_of_the_default_kind_and_the_current_one(bsr):
    b = Batch([300, 70], [40, 1], 2, 64, seed=9)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    want, lse = bsr.paged_attn(q, *b.where)
    for stream in (torch.cuda.current_stream(), torch.cuda.default_stream()):
        o, l2 = bsr.paged_attn(q, *b.where, stream=stream)
        assert torch.equal(o, want) and torch.equal(l2, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # and the default one from another
        o, l2 = bsr.paged_attn(q, *b.where, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(l2, lse)


def test_a_captured_call_on_another_stream(bsr):
    """A branch of a captured graph: outputs and workspace come from the
    graph's memory."""
    b = Batch([300, 70], [40, 1], 2, 64, seed=9)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    want, _ = bsr.paged_attn(q, *b.where)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        o, _ = bsr.paged_attn(q, *b.where, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        twice = o * 2
    for _ in range(3):
        o.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(twice, want * 2)
