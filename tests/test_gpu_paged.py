"""The paged cache and the attention over it, against the fp64 oracle.

Copies are compared bit for bit (BF16 moves, E4M3 by definition).

Attention tolerances (u = 2^-24).  With A = sum p |v| / sum p of the exact
probabilities and R the largest scale * sum_d |q_d k_d| of a visible key:
  * a logit is an FP32 sum of 128 exact products in some order, each addition
    off by at most one step even where the tensor core truncates: 128 * 2u R;
    its scaling and the subtraction of the row's reference add 8u R (the
    reference is at most R).  ds = (128 * 2 + 8) u R.
  * a probability carries 2 ds relative error in numerator and denominator
    together (first order, doubled below), 2^-22 of ex2 and one BF16 rounding
    for the matrix product, 2^-8 relative; FP32 sums over n keys and the
    merging of at most 64 partial sums (n + 64) 2u.  All of it times A.
  * the output is rounded to BF16 once: 2^-8 |o|.
  * lse: ds + (n + 64) 2u + 2^-21, and the logarithm and its scaling 4u |lse|.
"""

import math

import numpy as np
import pytest

import oracle as O
from oracle import paged as OP

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def bsr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_routed_gb300 as m

    m.load_library()
    return m


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Batch:
    """A ragged batch in a shuffled pool, with garbage wherever no token is."""

    def __init__(self, lens, news, H, page=64, kind="bf16", seed=0, spare=2, first_row=0, after=0, q_scale=1.0):
        g = np.random.default_rng(seed)
        self.lens, self.news, self.H, self.page, self.kind = list(lens), list(news), H, page, kind
        per = [-(-n // page) for n in lens]
        self.pages = sum(per) + spare
        width = max(per + [1]) + 1
        order = g.permutation(self.pages)
        table = np.full((len(lens), width), -7, dtype=np.int32)  # unused entries are invalid
        at = 0
        for s, n in enumerate(per):
            table[s, :n] = order[at:at + n]
            table[s, n:] = [-7, 2 ** 31 - 1][s % 2]
            at += n
        self.table_np = table
        self.starts = np.concatenate([[first_row], first_row + np.cumsum(self.news)]).astype(np.int32)
        self.rows = int(self.starts[-1]) + after
        self.table = torch.from_numpy(table).cuda()
        self.row_start = torch.from_numpy(self.starts).cuda()
        self.kv_len = torch.tensor(self.lens, dtype=torch.int32).cuda()
        # garbage: NaN in every slot that no token owns
        self.owned = np.zeros((self.pages, page), dtype=bool)
        for s, n in enumerate(lens):
            j = np.arange(n)
            self.owned[table[s, j // page], j % page] = True
        shape = (self.pages, H, page, 128)
        k, v = (g.standard_normal(shape).astype(np.float32) for _ in range(2))
        k += g.standard_normal((1, H, 1, 128)).astype(np.float32)
        v *= np.exp(g.standard_normal((self.pages, 1, page, 1))).astype(np.float32)
        own = torch.from_numpy(self.owned)[:, None, :, None]
        self.k, self.v, self.k_exp, self.v_exp = [], [], None, None
        vals, exps = [], []
        for x in (k, v):
            t = torch.from_numpy(x).bfloat16()
            if kind == "bf16":
                t = torch.where(own, t, torch.full_like(t, math.nan))
                vals.append((t.cuda(), t.double().numpy()))
                exps.append(None)
            else:
                f, e = torch.frexp(t.float().abs().amax(-1, keepdim=True))
                e = torch.where(f > 0.875, e - 8, e - 9).clamp(min=-126)
                code = (t.double() * torch.exp2(-e.double())).float().to(torch.float8_e4m3fn).view(torch.uint8)
                code = torch.where(own, code, torch.full_like(code, 127))
                byte = (e + 127).to(torch.uint8)[..., 0]
                byte = torch.where(own[..., 0].expand_as(byte), byte, torch.full_like(byte, 255))
                vals.append((code.view(torch.float8_e4m3fn).cuda(), OP.dequantise(code.numpy(), byte.numpy())))
                exps.append(byte.cuda())
        (self.k_pages, self.k64), (self.v_pages, self.v64) = vals
        self.k_exp, self.v_exp = exps

    @property
    def where(self):
        return self.k_pages, self.v_pages, self.table, self.row_start, self.kv_len

    @property
    def exps(self):
        return dict(k_exp=self.k_exp, v_exp=self.v_exp)


def check_attention(b, q, o, lse, causal=True, window=0, scale=None, filled=None):
    """Every row of every sequence within the bounds above; `filled`: what
    rows of no sequence must still hold."""
    q64 = q.double().cpu().numpy()
    og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
    worst = 0.0
    member = np.zeros(b.rows, dtype=bool)
    for s, n in enumerate(b.lens):
        rows = [r for r, _ in OP.positions(b.starts, b.kv_len.cpu().numpy(), s)]
        pos = [p for _, p in OP.positions(b.starts, b.kv_len.cpu().numpy(), s)]
        if not rows:
            continue
        member[rows] = True
        k, v = OP.gather(b.k64, b.table_np, s, n), OP.gather(b.v64, b.table_np, s, n)
        ro, rl, mass, reach = OP.paged_attention(q64[rows], k, v, pos, n, causal, window, scale)
        ds = (2 * 128 + 8) * U * reach
        tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (n + 64) * U)[..., None] * mass
        d = np.abs(og[rows] - ro)
        assert np.all(np.isfinite(og[rows])), s
        assert np.all(d <= tol), (s, d.max(), (d / np.maximum(tol, 1e-30)).max())
        worst = max(worst, float((d / np.maximum(tol, 1e-30)).max()))
        empty = np.isinf(rl)
        assert np.array_equal(lg[rows] == -np.inf, empty), s
        with np.errstate(invalid="ignore"):
            dl = np.where(empty, 0, np.abs(lg[rows] - rl))
        tl = ds + 2 * (n + 64) * U + 2.0 ** -21 + np.where(empty, 0, 4 * U * np.abs(np.where(empty, 0, rl)))
        assert np.all(dl <= tl), (s, dl.max())
    if filled is not None:
        assert np.all(og[~member] == filled) and np.all(lg[~member] == filled)
    return worst


def run_attention(bsr, b, Hq, seed=1, tight=True, **kw):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((b.rows, Hq, 128), generator=g).bfloat16().cuda() * 2
    o = torch.full((b.rows, Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.rows, Hq), 3.0, device="cuda")
    max_new = max(b.news) if tight else None
    ws = bsr.paged_workspace(q, b.k_pages, b.table, max_new)
    ws.fill_(255)  # scratch is the call's own business
    bsr.paged_attn(q, *b.where, max_new=max_new, **b.exps, o=o, lse=lse, ws=ws, **kw)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    return q, o, lse


# ---- copies

def rows_of(n, H, seed=0, strided=False):
    g = torch.Generator().manual_seed(seed)
    if strided:  # K and V as views of one projection's output, heads apart
        x = torch.randn((n, H, 3, 136), generator=g).bfloat16().cuda()
        return x[:, :, 1, :128], x[:, :, 2, :128]
    x = torch.randn((2, n, H, 128), generator=g).bfloat16().cuda()
    return x[0], x[1]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,H,lens,news,strided", [
    (16, 1, [1], [1], False),
    (64, 8, [64, 1, 65, 130], [1, 1, 1, 1], False),
    (32, 5, [0, 100, 33, 7], [0, 37, 33, 9], True),   # an empty sequence, and rows before its first token
    (128, 2, [257, 128], [200, 128], True),
    (64, 56, [70], [70], False),
])
def test_write_then_read(bsr, kind, page, H, lens, news, strided):
    b = Batch(lens, news, H, page, kind, first_row=2, after=3)
    k, v = rows_of(b.rows, H, strided=strided)
    before = [t.clone() for t in (b.k_pages, b.v_pages)]
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    bsr.cache_write(k, v, *b.where, **b.exps, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    expected = []
    for t, old in ((k, before[0]), (v, before[1])):
        tb = bits(t)
        raw = old.cpu().view(torch.uint8).numpy().copy()  # [pages, H, page, bytes]
        back = np.full((b.rows, H, 128), 7.0)
        for s in range(len(lens)):
            for r, p in OP.positions(b.starts, lens, s):
                if p < 0:
                    back[r] = 0.0
                    continue
                pg, sl = b.table_np[s, p // page], p % page
                for h in range(H):
                    if kind == "bf16":
                        raw[pg, h, sl] = tb[r, h].view(np.uint8)
                        back[r, h] = O.decode_bf16(tb[r, h])
                    else:
                        code, byte = OP.quantise_row(tb[r, h])
                        raw[pg, h, sl] = code
                        back[r, h] = OP.dequantise(code[None], np.array([byte]))[0]
        expected.append((raw, back))
    for t, (raw, _) in zip((b.k_pages, b.v_pages), expected):
        assert np.array_equal(t.cpu().view(torch.uint8).numpy(), raw)  # every other byte as it was
    out = [torch.full((b.rows, H, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bsr.cache_read(*b.where, **b.exps, k=out[0], v=out[1], ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    for t, (_, back) in zip(out, expected):
        assert np.array_equal(t.double().cpu().numpy(), back)


def test_quantised_extremes(bsr):
    """Zero rows, subnormals, the largest values, NaN and infinities."""
    x = torch.zeros((8, 1, 128), dtype=torch.float32)
    x[1, 0, 5] = 2.0 ** -133                      # the smallest BF16
    x[2, 0, :] = 3.3895e38                        # the largest
    x[3, 0, 0], x[3, 0, 1] = math.nan, 1.5
    x[4, 0, 0], x[4, 0, 1], x[4, 0, 2] = math.inf, -math.inf, -2.0
    x[5, 0, :] = -448.0
    x[6, 0, :] = 449.0                            # 448 in BF16's steps of 2: 448 or 450
    x[7, 0, :] = torch.linspace(-1, 1, 128)
    x = x.bfloat16().cuda()
    b = Batch([8], [8], 1, 16, "e4m3")
    bsr.cache_write(x, x, *b.where, **b.exps)
    codes = b.k_pages.cpu().view(torch.uint8).numpy()[b.table_np[0, 0], 0, :8]
    exps = b.k_exp.cpu().numpy()[b.table_np[0, 0], 0, :8]
    for r in range(8):
        want, byte = OP.quantise_row(bits(x)[r, 0])
        same = (codes[r] & 127 == 127) & (want & 127 == 127)  # any NaN
        assert exps[r] == byte and np.all(same | (codes[r] == want)), r
    k, _ = bsr.cache_read(*b.where, rows=8, **b.exps)
    assert k[3:5].isnan().all() and not k[:2].isnan().any() and not k[5:].isnan().any()


# ---- attention

RAGGED = ([1, 0, 63, 64, 65, 200, 129], [1, 0, 1, 1, 1, 1, 1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hq", [(1, 1), (2, 16), (8, 8), (3, 15), (1, 40)])
def test_single_tokens(bsr, kind, page, H, Hq):
    b = Batch(*RAGGED, H, page, kind, seed=H + Hq, after=2)
    q, o, lse = run_attention(bsr, b, Hq)
    check_attention(b, q, o, lse, filled=3.0)


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
])
@pytest.mark.parametrize("tight", [True, False])
def test_chunks(bsr, kind, lens, news, H, Hq, page, causal, window, tight):
    b = Batch(lens, news, H, page, kind, seed=len(lens) + window, first_row=1, after=1)
    q, o, lse = run_attention(bsr, b, Hq, tight=tight, causal=causal, window=window)
    check_attention(b, q, o, lse, causal, window, filled=3.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("lens,news,H,Hq,causal,window", [
    ([1500, 333, 81], [140, 60, 80], 1, 4, True, 200),   # windows begin inside pages and tiles
    ([1500, 333, 81], [140, 60, 80], 1, 4, False, 0),
    ([2600, 900], [40, 100], 2, 2, True, 0),             # units of few rows, cut many times, beside full ones
    ([2600, 900], [40, 600], 2, 2, True, 0),
    ([400, 17], [20, 3], 1, 40, True, 0),                # a row tile holds few tokens
    ([90, 170], [2, 3], 1, 300, True, 0),                # or less than one
])
def test_chunks_of_whole_page_runs(bsr, kind, page, lens, news, H, Hq, causal, window):
    b = Batch(lens, news, H, page, kind, seed=page + len(lens), after=1)
    q, o, lse = run_attention(bsr, b, Hq, causal=causal, window=window)
    check_attention(b, q, o, lse, causal, window, filled=3.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 150])
def test_long_context_is_split_and_joined(bsr, kind, news):
    b = Batch([9505, 40], [news, 1], 2, 64, kind, seed=5)
    q, o, lse = run_attention(bsr, b, 4)
    check_attention(b, q, o, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_sequences(bsr, kind):
    """More sequences than the work's scan looks at in one go, most of them
    without rows or tokens; in both forms."""
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(0, 40, 1100)]
    for most in (1, 30):
        news = [int(g.integers(0, most + 1)) if g.random() < 0.3 else 0 for _ in lens]
        news[700] = most
        b = Batch(lens, news, 1, 16, kind, seed=6)
        q, o, lse = run_attention(bsr, b, 4)
        check_attention(b, q, o, lse)
        k, v = rows_of(b.rows, 1)
        one = torch.empty(256, dtype=torch.uint8, device="cuda")
        bsr.cache_write(k, v, *b.where, **b.exps, ws=one)
        assert bsr.sparse_attn_last_device_status(one) == 0
        back, _ = bsr.cache_read(*b.where, rows=b.rows, **b.exps, ws=one)
        assert bsr.sparse_attn_last_device_status(one) == 0
        pos = np.array([p for s in range(len(lens)) for _, p in OP.positions(b.starts, lens, s)])
        there = torch.from_numpy(pos >= 0).cuda()
        assert not back[~there].any()
        if kind == "bf16":
            assert torch.equal(back[there], k[there])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_window_leaves_freed_pages_unread(bsr, kind):
    b = Batch([1000, 900], [3, 40], 2, 32, kind, seed=8)
    t = b.table.clone()
    t[0, : (1000 - 3 - 50) // 32] = -1     # pages below every row's window
    t[1, : (900 - 40 - 50) // 32] = 1 << 30
    b.table = t
    q, o, lse = run_attention(bsr, b, 4, window=50)
    check_attention(b, q, o, lse, True, 50)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,news,H,Hq,window", [
    ([100, 70], [3, 2], 2, 4, 0),          # few rows
    ([100, 300], [4, 3], 1, 4, 20),
    ([300, 150], [200, 90], 2, 4, 0),      # chunks
    ([500, 260], [257, 130], 1, 3, 33),
])
def test_odd_values_reach_only_the_rows_that_see_them(bsr, kind, lens, news, H, Hq, window):
    """NaN and infinities in K and V of tokens that only some rows of a tile
    see: the others' results are those of a cache without them."""
    for what in ("v nan", "v inf", "k nan", "v both"):
        b = Batch(lens, news, H, 64, kind, seed=3)
        bad = []
        for s, (n, m) in enumerate(zip(lens, news)):  # the newest token, one in the middle of the new ones, one old one
            bad += [(s, n - 1), (s, n - 1 - m // 2)] + ([(s, n - m - 30)] if window else [])
        for s, j in bad:
            pg, sl = b.table_np[s, j // 64], j % 64
            t, t64, e = (b.k_pages, b.k64, b.k_exp) if what[0] == "k" else (b.v_pages, b.v64, b.v_exp)
            if kind == "e4m3":
                e[pg, :, sl] = 255
                t64[pg, :, sl] = math.nan
                continue
            for d, x in {"nan": [(5, math.nan)], "inf": [(5, math.inf), (9, -math.inf)],
                         "both": [(d, math.nan if d % 3 else math.inf) for d in range(0, 128, 7)]}[what[2:]]:
                t[pg, :, sl, d] = x
                t64[pg, :, sl, d] = x
        q, o, lse = run_attention(bsr, b, Hq, window=window)
        og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
        seen = []
        for s, n in enumerate(lens):
            rows, pos = zip(*OP.positions(b.starts, lens, s))
            k, v = OP.gather(b.k64, b.table_np, s, n), OP.gather(b.v64, b.table_np, s, n)
            with np.errstate(invalid="ignore"):
                ro, rl, mass, reach = OP.paged_attention(q.double().cpu().numpy()[list(rows)], k, v, pos, n, True, window)
            got = og[list(rows)]
            fine = np.isfinite(ro)
            assert np.array_equal(fine, np.isfinite(got)), (what, s)
            assert np.array_equal(np.isnan(ro), np.isnan(got)) and np.array_equal(ro[np.isinf(ro)], got[np.isinf(ro)])
            mass = np.where(np.isfinite(mass), mass, 0)
            reach = np.where(np.isfinite(reach), reach, 0)
            ds = (2 * 128 + 8) * U * reach
            tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (n + 64) * U)[..., None] * mass
            with np.errstate(invalid="ignore"):
                assert np.all(np.abs(got - ro)[fine] <= tol[fine]), (what, s)
            assert np.array_equal(np.isnan(rl), np.isnan(lg[list(rows)]))
            seen.append(fine.reshape(-1))
        seen = np.concatenate(seen)
        assert seen.any() and not seen.all()  # both kinds of rows are there


def test_scales(bsr):
    b = Batch([333, 64], [20, 1], 2, 64, seed=3)
    for scale in (1e-6, 0.05, 3.0):
        q, o, lse = run_attention(bsr, b, 4, scale=scale)
        check_attention(b, q, o, lse, scale=scale)


def test_strided_queries(bsr):
    b = Batch([200, 90], [70, 1], 2, 64, seed=4)
    x = torch.randn((b.rows, 3, 4, 136), device="cuda").bfloat16()
    q = x[:, 1, :, :128]
    o, lse = bsr.paged_attn(q, *b.where)
    check_attention(b, q, o, lse)
    same = torch.randn((1, 1, 128), device="cuda").bfloat16().expand(b.rows, 4, 128)
    o, lse = bsr.paged_attn(same, *b.where)
    check_attention(b, same, o, lse)


def test_rising_logits_move_the_reference(bsr):
    """Keys that grow along the context: the running maximum moves all the time."""
    for news in (1, 40):
        b = Batch([1500], [news], 1, 64, seed=6)
        ramp = torch.zeros_like(b.k_pages)
        for j in range(1500):
            ramp[b.table_np[0, j // 64], 0, j % 64] = 0.02 * j
        b.k_pages = ramp
        b.k64 = ramp.double().cpu().numpy()
        q = torch.ones((b.rows, 2, 128), dtype=torch.bfloat16, device="cuda")
        o, lse = bsr.paged_attn(q, *b.where)
        check_attention(b, q, o, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(bsr, kind):
    """Tokens in the last pages of a pool of more than 2^32 bytes a tensor."""
    H, page = 2, 64
    pages = (1 << 32) // (H * page * (256 if kind == "bf16" else 128)) + 40
    k, v, ke, ve = bsr.paged_cache(pages, H, page, kind)
    n = 150
    table = torch.tensor([[pages - 1, pages - 3, 5]], dtype=torch.int32, device="cuda")
    rs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kl = torch.tensor([n], dtype=torch.int32, device="cuda")
    xk, xv = rows_of(n, H, seed=2)
    bsr.cache_write(xk, xv, k, v, table, rs, kl, k_exp=ke, v_exp=ve)
    rk, rv = bsr.cache_read(k, v, table, rs, kl, rows=n, k_exp=ke, v_exp=ve)
    for x, y in ((xk, rk), (xv, rv)):
        if kind == "bf16":
            assert torch.equal(x, y)
        else:
            amax = x.float().abs().amax(-1, keepdim=True)
            assert ((x.float() - y.float()).abs() <= torch.maximum(2.0 ** -4 * x.float().abs(), 2.0 ** -10 * amax / 224)).all()
    for m in (1, n):
        q = torch.randn((m, 4, 128), device="cuda").bfloat16()
        r = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        o, lse = bsr.paged_attn(q, k, v, table, r, kl, max_new=m, k_exp=ke, v_exp=ve)
        pos = list(range(n - m, n))
        ro, rl, mass, reach = OP.paged_attention(q.double().cpu().numpy(), rk.double().cpu().numpy(),
                                                 rv.double().cpu().numpy(), pos, n)
        ds = (2 * 128 + 8) * U * reach
        tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (n + 64) * U)[..., None] * mass
        assert np.all(np.abs(o.double().cpu().numpy() - ro) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - rl) <= ds + 2 * (n + 64) * U + 2.0 ** -21 + 4 * U * np.abs(rl))


# ---- what the device refuses

def test_bad_pages_are_reported_and_not_read(bsr):
    for kind in ("bf16", "e4m3"):
        for news in (1, 30):
            b = Batch([200, 90], [news, 1], 2, 64, kind, seed=4)
            for bad in (-1, b.pages, 2 ** 31 - 1, -2 ** 31):
                t = b.table.clone()
                t[0, 3] = bad  # the page of the first sequence's newest tokens
                q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
                ws = bsr.paged_workspace(q, b.k_pages, t, news)
                o, lse = bsr.paged_attn(q, b.k_pages, b.v_pages, t, b.row_start, b.kv_len, max_new=news, ws=ws, **b.exps)
                assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL
                one = torch.empty(256, dtype=torch.uint8, device="cuda")
                k, v = rows_of(b.rows, 2)
                before = b.k_pages.clone()
                bsr.cache_read(b.k_pages, b.v_pages, t, b.row_start, b.kv_len, rows=b.rows, ws=one, **b.exps)
                assert bsr.sparse_attn_last_device_status(one) == bsr.SA_EINVAL
                bsr.cache_write(k, v, b.k_pages, b.v_pages, t, b.row_start, b.kv_len, ws=one, **b.exps)
                assert bsr.sparse_attn_last_device_status(one) == bsr.SA_EINVAL
                b.k_pages.copy_(before)
                # the status is the call's own: a good call on the same workspace clears it
                bsr.paged_attn(q, *b.where, max_new=news, ws=ws, **b.exps)
                assert bsr.sparse_attn_last_device_status(ws) == 0


@pytest.mark.parametrize("starts,lens,max_new", [
    ([0, 5, 3], [200, 90], None),          # not ascending
    ([0, 5, 99], [200, 90], None),         # past the rows
    ([-1, 1, 2], [200, 90], None),
    ([0, 1, 2], [-1, 90], None),
    ([0, 1, 2], [200, 100000], None),      # more tokens than the table has pages for
    ([0, 4, 5], [200, 90], 3),             # more rows than max_new
])
def test_bad_batches_are_reported(bsr, starts, lens, max_new):
    b = Batch([200, 90], [4, 1], 2, 64, seed=4)
    rs = torch.tensor(starts, dtype=torch.int32, device="cuda")
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((5, 4, 128), device="cuda").bfloat16()
    for mn in ([max_new] if max_new else [None, 1]):
        ws = bsr.paged_workspace(q, b.k_pages, b.table, mn)
        bsr.paged_attn(q, b.k_pages, b.v_pages, b.table, rs, kl, max_new=mn, ws=ws)
        assert bsr.sparse_attn_last_device_status(ws) == bsr.SA_EINVAL
    if max_new is None:
        one = torch.empty(256, dtype=torch.uint8, device="cuda")
        bsr.cache_read(b.k_pages, b.v_pages, b.table, rs, kl, rows=5, ws=one)
        assert bsr.sparse_attn_last_device_status(one) == bsr.SA_EINVAL
        k, v = rows_of(5, 2)
        bsr.cache_write(k, v, b.k_pages, b.v_pages, b.table, rs, kl, ws=one)
        assert bsr.sparse_attn_last_device_status(one) == bsr.SA_EINVAL


def test_refusals_of_the_python_layer(bsr):
    b = Batch([200, 90], [4, 1], 2, 64, seed=4)
    q = torch.randn((b.rows, 4, 128), device="cuda").bfloat16()
    call = lambda q=q, **kw: bsr.paged_attn(q, *b.where, **kw)  # noqa: E731
    with pytest.raises(ValueError):
        call(q=q[:, :3])
    with pytest.raises(TypeError):
        call(q=q.half())
    with pytest.raises(ValueError):
        call(q=q.cpu())
    with pytest.raises(ValueError):
        call(window=-1)
    with pytest.raises(ValueError):
        call(window=5, causal=False)
    with pytest.raises(ValueError):
        call(max_new=-1)
    with pytest.raises(ValueError):
        call(o=torch.empty((b.rows, 4, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        call(lse=torch.empty((b.rows, 4), dtype=torch.float64, device="cuda"))
    with pytest.raises(bsr.SparseAttnError):
        call(ws=torch.empty(255, dtype=torch.uint8, device="cuda"))
    with pytest.raises(bsr.SparseAttnError):
        call(scale=math.inf)
    with pytest.raises(bsr.SparseAttnError):
        call(scale=-0.1)
    with pytest.raises(ValueError):
        call(k_exp=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        bsr.paged_attn(q, b.k_pages, b.v_pages, b.table.long(), b.row_start, b.kv_len)
    with pytest.raises(ValueError):
        bsr.paged_attn(q, b.k_pages, b.v_pages, b.table, b.row_start[:-1], b.kv_len)
    with pytest.raises(ValueError):
        bsr.paged_attn(q, b.k_pages, b.v_pages[:1], b.table, b.row_start, b.kv_len)
    with pytest.raises(ValueError):
        bsr.cache_write(q[:, :2, :64], q[:, :2, :64], *b.where)
    with pytest.raises(ValueError):
        bsr.cache_read(*b.where)


def test_nothing_to_do(bsr):
    k, v, _, _ = bsr.paged_cache(4, 2, 16)
    empty = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for seqs in (0, 3):
        batch = (torch.empty((seqs, 2), **i32), torch.zeros(seqs + 1, **i32), torch.zeros(seqs, **i32))
        ws = bsr.paged_workspace(empty, k, batch[0]).fill_(255)
        o, lse = bsr.paged_attn(empty, k, v, *batch, ws=ws)
        assert o.shape == (0, 4, 128) and bsr.sparse_attn_last_device_status(ws) == 0
        bsr.cache_write(empty[:, :2], empty[:, :2], k, v, *batch)
        assert bsr.cache_read(k, v, *batch, rows=0)[0].shape == (0, 2, 128)
    # rows, but of no sequence
    q = torch.ones((3, 4, 128), dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 5.0)
    bsr.paged_attn(q, k, v, torch.empty((0, 2), **i32), torch.zeros(1, **i32), torch.zeros(0, **i32), o=o)
    assert (o == 5).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 300])
def test_a_wait_that_gives_up_is_reported(bsr, kind, news):
    """The testing hook makes every pipeline wait a single probe: the call
    records the timeout and ends by itself, the next one is as ever."""
    from block_sparse_routed_gb300 import _native

    b = Batch([900, 70], [news, 1], 2, 64, kind, seed=9)
    q, o, lse = run_attention(bsr, b, 4)
    ws = bsr.paged_workspace(q, b.k_pages, b.table, news)
    prev = _native.sparse_attn_set_single_probe_waits(True)
    try:
        statuses = []
        for _ in range(5):  # a single probe almost surely comes too early
            bsr.paged_attn(q, *b.where, max_new=news, **b.exps, ws=ws)
            statuses.append(bsr.sparse_attn_last_device_status(ws))
            if statuses[-1] == bsr.SA_ETIMEOUT:
                break
    finally:
        _native.sparse_attn_set_single_probe_waits(bool(prev))
    assert bsr.SA_ETIMEOUT in statuses
    o2, l2 = bsr.paged_attn(q, *b.where, max_new=news, **b.exps, ws=ws)
    assert bsr.sparse_attn_last_device_status(ws) == 0
    assert torch.equal(o, o2) and torch.equal(lse, l2)


# ---- streams, graphs, repeatability

def test_bitwise_repeatable(bsr):
    for news in (1, 33):
        b = Batch([3000, 70, 1200], [news, 1, news], 2, 64, "e4m3", seed=9)
        q, o, lse = run_attention(bsr, b, 8)
        for _ in range(3):
            o2, l2 = bsr.paged_attn(q, *b.where, max_new=news, **b.exps)
            assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_another_stream(bsr):
    b = Batch([3000, 70], [40, 1], 2, 64, seed=9)
    q, o, lse = run_attention(bsr, b, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = bsr.paged_attn(q, *b.where, max_new=40, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    with torch.cuda.stream(side):
        o3, _ = bsr.paged_attn(q, *b.where, max_new=40)
    side.synchronize()
    assert torch.equal(o, o3)


def test_captured_decoding_steps(bsr):
    """One captured step (write, attend) replayed while lengths, pages and
    inputs change in place; two graphs share one workspace, one after the other."""
    H, Hq, page, S = 2, 8, 16, 3
    k, v, ke, ve = bsr.paged_cache(S * 8, H, page, "e4m3")
    g = torch.Generator().manual_seed(0)
    perm = torch.randperm(S * 8, generator=g).to(torch.int32).reshape(S, 8)
    table = perm.cuda()
    rs = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    kl = torch.zeros(S, dtype=torch.int32, device="cuda")
    xk, xv = (torch.zeros((S, H, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qs = [torch.zeros((S, Hq, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    outs = [(torch.zeros_like(q), torch.zeros((S, Hq), device="cuda")) for q in qs]
    ws = bsr.paged_workspace(qs[0], k, table, 1)

    def step(i):
        if i == 0:
            bsr.cache_write(xk, xv, k, v, table, rs, kl, k_exp=ke, v_exp=ve)
        bsr.paged_attn(qs[i], k, v, table, rs, kl, max_new=1, k_exp=ke, v_exp=ve, o=outs[i][0], lse=outs[i][1], ws=ws)

    graphs = []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(i)
        graphs.append(gr)
    hist_k, hist_v = [], []
    for t in range(40):
        xk.copy_(torch.randn((S, H, 128), generator=g).bfloat16())
        xv.copy_(torch.randn((S, H, 128), generator=g).bfloat16())
        for q in qs:
            q.copy_(torch.randn((S, Hq, 128), generator=g).bfloat16() * 2)
        kl.add_(1)
        graphs[0].replay()
        graphs[1].replay()
        back = bsr.cache_read(k, v, table, rs, kl, rows=S, k_exp=ke, v_exp=ve)
        hist_k.append(back[0].double().cpu().numpy())
        hist_v.append(back[1].double().cpu().numpy())
        if t % 13 in (0, 12):
            for i in range(2):
                q64 = qs[i].double().cpu().numpy()
                for s in range(S):
                    kk, vv = np.stack(hist_k)[:, s], np.stack(hist_v)[:, s]
                    ro, rl, mass, reach = OP.paged_attention(q64[s:s + 1], kk, vv, [t], t + 1)
                    ds = (2 * 128 + 8) * U * reach
                    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (t + 65) * U)[..., None] * mass
                    assert np.all(np.abs(outs[i][0][s:s + 1].double().cpu().numpy() - ro) <= tol)


# ---- together, and with what the library had

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_prompt_in_chunks_equals_the_prompt_at_once(bsr, kind):
    H, Hq, n, page = 2, 6, 333, 32
    xk, xv = rows_of(n, H, seed=11)
    q = torch.randn((n, Hq, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(11, device="cuda").to(torch.int32)[None]
    results = []
    for cuts in ([n], [100, 1, 64, 1, 167]):
        k, v, ke, ve = bsr.paged_cache(11, H, page, kind)
        at, parts = 0, []
        for m in cuts:
            rs, kl = torch.tensor([0, m], **i32), torch.tensor([at + m], **i32)
            bsr.cache_write(xk[at:at + m], xv[at:at + m], k, v, table, rs, kl, k_exp=ke, v_exp=ve)
            parts.append(bsr.paged_attn(q[at:at + m], k, v, table, rs, kl, k_exp=ke, v_exp=ve))
            at += m
        results.append([torch.cat(x) for x in zip(*parts)])
    back = bsr.cache_read(k, v, table, torch.tensor([0, n], **i32), torch.tensor([n], **i32), rows=n, k_exp=ke, v_exp=ve)
    k64, v64 = (t.double().cpu().numpy() for t in back)
    ro, rl, mass, reach = OP.paged_attention(q.double().cpu().numpy(), k64, v64, list(range(n)), n)
    ds = (2 * 128 + 8) * U * reach
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * ds + 2.0 ** -21 + 2 * (n + 64) * U)[..., None] * mass
    for o, lse in results:
        assert np.all(np.abs(o.double().cpu().numpy() - ro) <= tol)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_cached_context_through_the_routed_attention(bsr, kind):
    """cache_read's output is what sparse_attn takes; with every block listed
    it computes what paged_attn computes with causal=False."""
    H, n = 2, 640
    b = Batch([n], [n], H, 64, kind, seed=12)
    q = torch.randn((n, H, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    k, v = bsr.cache_read(*b.where, rows=n, **b.exps)
    p = bsr.Params(T=n, H=H, video_tokens=n, topk_ratio=1.0, radius=1)
    ref = bsr.sparse_attn(p, q[None], k[None], v[None])[0]
    o, lse = bsr.paged_attn(q, *b.where, causal=False, **b.exps)
    check_attention(b, q, o, lse, causal=False)
    check_attention(b, q, ref, lse, causal=False)
