"""Cases of the paged key/value cache and of the attention that reads it.

Three operators, with one description of a batch for all of them.  A cache is
``k_pages`` and ``v_pages`` [pages, H, page_size, 128], BF16, or E4M3 with one
power-of-two scale a row, held as its exponent ``k_exp`` and ``v_exp`` (uint8
[pages, H, page_size], value e stands for 2^(e - 127)).  Sequence s has
``kv_len[s]`` tokens, token j in slot j % page_size of page
``table[s, j // page_size]``, and the rows ``row_start[s] .. row_start[s + 1]``
of a packed tensor are its last tokens: with n rows, row i is the token at
position kv_len[s] - n + i.

* write: rows of K and V go into the cache, quantised on the way (E4M3).
* read: the inverse, rows of K and V as BF16.
* attn: rows of Q attend to the cached keys of their sequence, up to their own
  position (causal), the last ``window`` of these, or all of them; Hq query
  heads share H key heads in order.  One token a sequence is decoding, more
  are a chunk.
"""

import math
import random

import torch

own = False

D = 128

# Head counts, clip lengths and context lengths are those of the benchmark's
# workloads (tiny, 8k, h3, 32k, 64k): 2, 24, 40 and 56 heads, 1152 to 67608
# tokens; grouped key heads where a model serves single tokens.
_LISTED = [
    # every decoding step stores one token of each of 32 sequences
    dict(name="write, one token each", op="write", kind="e4m3", page=64, seqs=32, hq=8, h=8, new=1, lo=700, hi=8704),
    # a finished clip's K and V go into the cache in one call (h3: 9505 tokens, 56 heads)
    dict(name="write, a clip", op="write", kind="e4m3", page=64, seqs=1, hq=56, h=56, new=9505, lo=9505, hi=9505),
    # four short contexts handed back to an operator that wants packed tensors
    dict(name="read, short contexts", op="read", kind="e4m3", page=16, seqs=4, hq=2, h=2, new=1152, lo=77, hi=1152),
    # a long context handed back (64k: 67608 tokens, 24 heads)
    dict(name="read, a long context", op="read", kind="e4m3", page=64, seqs=1, hq=24, h=24, new=67608, lo=67608, hi=67608),
    # one user, short context: the latency of a call
    dict(name="decode, one sequence", op="attn", kind="bf16", page=64, seqs=1, hq=8, h=2, new=1, lo=1152, hi=1152, mask="causal", window=0),
    # a full decoding batch of ragged contexts
    dict(name="decode, a batch", op="attn", kind="bf16", page=64, seqs=64, hq=40, h=8, new=1, lo=512, hi=33792, mask="causal", window=0),
    # the same, over a quantised cache with smaller pages
    dict(name="decode, quantised", op="attn", kind="e4m3", page=32, seqs=96, hq=56, h=8, new=1, lo=512, hi=33792, mask="causal", window=0),
    # several drafted tokens a sequence are checked at once, with a sliding window
    dict(name="few tokens, window", op="attn", kind="e4m3", page=64, seqs=16, hq=24, h=8, new=4, lo=300, hi=8704, mask="causal", window=4096),
    # a prompt that is taken in chunks: 2048 new tokens behind a long context
    dict(name="chunk, long context", op="attn", kind="bf16", page=64, seqs=1, hq=40, h=8, new=2048, lo=33792, hi=33792, mask="causal", window=0),
    # a video chunk attends both ways to itself and to the cached clip
    dict(name="chunk, video", op="attn", kind="e4m3", page=64, seqs=1, hq=56, h=56, new=1320, lo=9505, hi=9505, mask="all", window=0),
    # one step of a server: some sequences bring a chunk, others a single token
    dict(name="mixed batch", op="attn", kind="bf16", page=16, seqs=7, hq=24, h=8, new=777, lo=900, hi=8704, mask="causal", window=0),
    # a whole prompt at once, nothing cached before it
    dict(name="whole prompt", op="attn", kind="bf16", page=64, seqs=1, hq=24, h=24, new=8704, lo=8704, hi=8704, mask="causal", window=0),
]


def listed():
    return [dict(c) for c in _LISTED]


def _spread(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def _lengths(case):
    """(tokens, new rows) of each sequence: a plain function of the case."""
    rng = random.Random(1009 * case["seqs"] + 31 * case["new"] + case["lo"] + 7 * case["hi"])
    n = case["seqs"]
    lens = [case["hi"]] + [_spread(rng, case["lo"], case["hi"]) for _ in range(n - 1)]
    news = [case["new"]] + [_spread(rng, 1, case["new"]) for _ in range(n - 1)]
    if case["op"] == "read":  # whole contexts
        news = lens
    return lens, [min(a, b) for a, b in zip(news, lens)]


def _spans(case):
    """(seen key-row pairs, keys read) summed over the sequences, of one head."""
    pairs = keys = 0
    for n, m in zip(*_lengths(case)):
        if case["mask"] == "all":
            pairs, keys = pairs + n * m, keys + n
        else:
            w = case["window"] or n
            pairs += sum(min(p + 1, w) for p in range(n - m, n))
            keys += n - max(0, n - m - w + 1)
    return pairs, keys


def work(case):
    lens, news = _lengths(case)
    rows, h, hq = sum(news), case["h"], case["hq"]
    cached = 2 * D if case["kind"] == "bf16" else D + 1  # bytes of a cached row
    if case["op"] != "attn":
        return {"bytes": 2 * rows * h * (2 * D + cached), "flops": 0}
    pairs, keys = _spans(case)
    return {"bytes": 2 * keys * h * cached + rows * hq * (4 * D + 4), "flops": 4 * D * hq * pairs}


def _padded(case):
    """Scores of the plain form, which pads every sequence to the longest."""
    return case["seqs"] * case["new"] * case["hq"] * case["hi"] if case["op"] == "attn" else 0


def draw(rng):
    top = {"write": 2.6e8, "read": 1.2e9, "attn": 1.6e9}
    while True:
        op = rng.choice(["write", "read", "attn", "attn", "attn", "attn"])
        h = rng.choice([1, 2, 8, 8, 24, 40])
        c = dict(op=op, kind=rng.choice(["bf16", "e4m3"]), page=rng.choice([16, 32, 64, 128]),
                 seqs=_spread(rng, 1, 96), hq=h * rng.choice([1, 1, 3, 4, 5, 7, 8]), h=h)
        c["hi"] = _spread(rng, 100, 33792)
        c["lo"] = _spread(rng, 1, c["hi"])
        c["new"] = rng.choice([1, _spread(rng, 2, 8), _spread(rng, 9, 8704)])
        if op == "attn":
            c["mask"] = rng.choice(["causal", "causal", "all"])
            c["window"] = _spread(rng, 16, 8192) if c["mask"] == "causal" and rng.random() < 0.3 else 0
            if c["hq"] > 64 or _padded(c) > 2e9:
                continue
        else:
            c["hq"] = h
        w = work(c)
        if 2e5 <= w["bytes"] <= top[op] and w["flops"] <= 9e11 and sum(_lengths(c)[0]) * h <= 1.5e7:
            return c


def _two(e):
    """2^e in 32 bits, exact (-126 <= e <= 127)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """E4M3 codes and exponents of rows: the smallest 2^e that brings the row's largest magnitude to 448 or less."""
    x = x.float()
    f, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = torch.where(f > 0.875, e - 8, e - 9).clamp(min=-126)
    return (x * _two(-e)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).squeeze(-1)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(dev).manual_seed(seed)
    lens, news = _lengths(case)
    h, ps, bf = case["h"], case["page"], torch.bfloat16
    width = -(-max(lens) // ps)
    pages = [-(-n // ps) for n in lens]
    total = sum(pages) + 3  # a few pages of the pool are free
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32)
    at = 0
    table = table.to(dev)
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    rows = starts[-1]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=bf)

    st = dict(op=case["op"], page=ps, new=max(news), table=table, rows=rows,
              row_start=torch.tensor(starts, dtype=torch.int32, device=dev),
              kv_len=torch.tensor(lens, dtype=torch.int32, device=dev), k_exp=None, v_exp=None)
    # keys around a mean of their head, values of uneven size from token to token
    if case["op"] == "write":
        kv = [normal(total, h, ps, D), normal(total, h, ps, D)]
        qkv = normal(rows, 3, h, D)  # the projection's output: K and V are strided views of it
        qkv[:, 1] += normal(h, D)
        qkv[:, 2] *= torch.exp(normal(rows, 1, 1))
        st["k"], st["v"] = qkv[:, 1], qkv[:, 2]
    else:
        kv = [normal(total, h, ps, D) + normal(h, 1, D), normal(total, h, ps, D) * torch.exp(normal(total, 1, ps, 1))]
    if case["kind"] == "e4m3":
        kv[0], st["k_exp"] = _quantise(kv[0])
        kv[1], st["v_exp"] = _quantise(kv[1])
    st["k_pages"], st["v_pages"] = kv
    if case["op"] == "attn":
        st["q"] = 2.0 * normal(rows, case["hq"], D)
        st["causal"], st["window"] = case["mask"] == "causal", case["window"]
        st["o"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((rows, case["hq"]), dtype=torch.float32, device=dev)
    elif case["op"] == "read":
        st["k"] = torch.zeros((rows, h, D), dtype=bf, device=dev)
        st["v"] = torch.zeros_like(st["k"])
    return st


def _rows(st):
    """Sequence and position of every row."""
    r = torch.arange(st["rows"], device=st["table"].device)
    s = torch.searchsorted(st["row_start"][1:], r, right=True)
    n = st["row_start"][1:] - st["row_start"][:-1]
    return s, r - st["row_start"][s], (st["kv_len"] - n)[s] + r - st["row_start"][s]


def _plain_write(st):
    s, _, pos = _rows(st)
    page, slot = st["table"][s, pos // st["page"]].long(), pos % st["page"]
    if st["k_exp"] is None:
        st["k_pages"][page, :, slot] = st["k"]
        st["v_pages"][page, :, slot] = st["v"]
        return st["k_pages"], st["v_pages"]
    (kc, ke), (vc, ve) = _quantise(st["k"]), _quantise(st["v"])
    # indexed stores move the codes as bytes
    st["k_pages"].view(torch.uint8)[page, :, slot] = kc.view(torch.uint8)
    st["v_pages"].view(torch.uint8)[page, :, slot] = vc.view(torch.uint8)
    st["k_exp"][page, :, slot] = ke
    st["v_exp"][page, :, slot] = ve
    return st["k_pages"], st["v_pages"], st["k_exp"], st["v_exp"]


def _values(pages, exp):
    """What cached rows stand for, in 32 bits."""
    x = pages.float()
    return x if exp is None else x * _two(exp.int().unsqueeze(-1) - 127)


def _plain_read(st):
    s, _, pos = _rows(st)
    page, slot = st["table"][s, pos // st["page"]].long(), pos % st["page"]
    if st["k_exp"] is None:
        return st["k_pages"][page, :, slot], st["v_pages"][page, :, slot]
    k = st["k_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
    v = st["v_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
    return (_values(k, st["k_exp"][page, :, slot]).to(torch.bfloat16),
            _values(v, st["v_exp"][page, :, slot]).to(torch.bfloat16))


def _padded_cache(pages, exp, table):
    """[sequences, heads, tokens, 128] of every sequence's pages."""
    t = table.long()
    x = pages[t] if exp is None else pages.view(torch.uint8)[t].view(pages.dtype)
    x = _values(x, None if exp is None else exp[t])
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attn(st):
    q, table, kv_len = st["q"], st["table"], st["kv_len"]
    s, i, pos = _rows(st)
    n_seq, hq, h = table.shape[0], q.shape[1], st["k_pages"].shape[1]
    k = _padded_cache(st["k_pages"], st["k_exp"], table)
    v = _padded_cache(st["v_pages"], st["v_exp"], table)
    qp = torch.zeros((n_seq, st["new"], hq, D), dtype=torch.float32, device=q.device)
    qp[s, i] = q.float()
    at = torch.zeros((n_seq, st["new"]), dtype=torch.int64, device=q.device)
    at[s, i] = pos
    # rows of one key head: (new token, query head of the group)
    qp = qp.unflatten(2, (h, hq // h)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = qp @ k.transpose(-1, -2)
    x *= 1.0 / math.sqrt(D)
    j = torch.arange(k.shape[2], device=q.device)
    seen = (j < kv_len[:, None, None]).expand(-1, st["new"], -1)
    if st["causal"]:
        seen = seen & (j <= at[..., None])
    if st["window"]:
        seen = seen & (j > at[..., None] - st["window"])
    seen = seen.unsqueeze(1).unsqueeze(3).expand(-1, -1, -1, hq // h, -1).flatten(2, 3)
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = x @ v
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log()).squeeze(-1)
    # back to packed rows
    o = o.unflatten(2, (st["new"], hq // h)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.unflatten(2, (st["new"], hq // h)).permute(0, 2, 1, 3).flatten(2, 3)
    return o[s, i].to(q.dtype), lse[s, i]


def run(state):
    st = state
    if own:
        import block_sparse_routed_gb300 as bsr

        batch = (st["table"], st["row_start"], st["kv_len"])
        if st["op"] == "write":
            bsr.cache_write(st["k"], st["v"], st["k_pages"], st["v_pages"], *batch, k_exp=st["k_exp"], v_exp=st["v_exp"])
            if st["k_exp"] is None:
                return st["k_pages"], st["v_pages"]
            return st["k_pages"], st["v_pages"], st["k_exp"], st["v_exp"]
        if st["op"] == "read":
            return bsr.cache_read(st["k_pages"], st["v_pages"], *batch, k_exp=st["k_exp"], v_exp=st["v_exp"], k=st["k"], v=st["v"])
        if "ws" not in st:  # a server keeps one workspace
            st["ws"] = bsr.paged_workspace(st["q"], st["k_pages"], st["table"], max_new=st["new"])
        return bsr.paged_attn(st["q"], st["k_pages"], st["v_pages"], *batch, max_new=st["new"], causal=st["causal"],
                              window=st["window"], k_exp=st["k_exp"], v_exp=st["v_exp"], o=st["o"], lse=st["lse"], ws=st["ws"])
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn}[st["op"]](st)


def _exact_rows(pages, exp, page, slot):
    """Cached rows [n, H, 128] in 64 bits."""
    if exp is None:
        return pages[page, :, slot].double()
    code = pages.view(torch.uint8)[page, :, slot].int()
    m, e = (code & 7).double(), (code >> 3) & 15
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e.double() - 7))
    two = torch.exp2(exp[page, :, slot].double() - 127)
    return torch.where(code >= 128, -mag, mag) * two.unsqueeze(-1)


def _nearest_e4m3(x):
    """The nearest value of the format, ties to even, of doubles up to 448 in size."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    lens, news = _lengths(case)
    ps, table = case["page"], st["table"].long()
    if case["op"] == "write":
        outs = []
        for name in ("k", "v"):
            pages, exp = st[name + "_pages"].double(), st[name + "_exp"]
            r0 = 0
            for s, (n, m) in enumerate(zip(lens, news)):
                x = st[name][r0:r0 + m].double()
                r0 += m
                j = torch.arange(n - m, n, device=x.device)
                page, slot = table[s, j // ps], j % ps
                if exp is not None:
                    most = x.abs().amax(-1) / 448
                    e = torch.round(torch.log2(most))  # within one of it, then the definition
                    e = torch.where(most > torch.exp2(e), e + 1, torch.where(most <= torch.exp2(e - 1), e - 1, e)).clamp(min=-126)
                    x = _nearest_e4m3(x / torch.exp2(e).unsqueeze(-1))
                    exp[page, :, slot] = (e + 127).to(torch.uint8)
                pages[page, :, slot] = x
            outs.append((pages, exp))
        (k, ke), (v, ve) = outs
        return (k, v) if ke is None else (k, v, ke, ve)
    ks, vs, os, ls = [], [], [], []
    r0 = 0
    for s, (n, m) in enumerate(zip(lens, news)):
        j = torch.arange(n, device=table.device)
        page, slot = table[s, j // ps], j % ps
        k = _exact_rows(st["k_pages"], st["k_exp"], page, slot)
        v = _exact_rows(st["v_pages"], st["v_exp"], page, slot)
        if case["op"] == "read":
            ks.append(k)
            vs.append(v)
            continue
        q = st["q"][r0:r0 + m].double()
        r0 += m
        p = torch.arange(n - m, n, device=table.device)[:, None]
        if case["mask"] == "all":
            hidden = torch.zeros((m, n), dtype=torch.bool, device=table.device)
        else:
            hidden = j[None] > p
            if case["window"]:
                hidden |= j[None] <= p - case["window"]
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
        for head in range(case["hq"]):
            kh = head // (case["hq"] // case["h"])
            x = torch.mm(q[:, head], k[:, kh].T) / math.sqrt(D)
            x[hidden] = -math.inf
            lse[:, head] = torch.logsumexp(x, 1)
            o[:, head] = torch.mm(torch.exp(x - lse[:, head, None]), v[:, kh])
        os.append(o)
        ls.append(lse)
    if case["op"] == "read":
        return torch.cat(ks), torch.cat(vs)
    return torch.cat(os), torch.cat(ls)
