"""Cases of three operators over a paged key/value cache that many sequences fill.

They share the batch of the cache's other calls (``k_pages``, ``v_pages`` [pages, H, page_size, 128] in BF16, or E4M3
with exponents ``k_exp``, ``v_exp``; ``table``, ``row_start``, ``kv_len``): the rows of a sequence are its last tokens.

* prefix: attention of the rows of q when the sequences ``group_start[g] .. group_start[g + 1]`` begin with the same
  ``prefix_len[g]`` tokens, whose whole pages they share. The prefix is read once for all rows of its group.
* weigh: attention weight that the cached keys received. ``weights`` [pages, H, page_size] takes, for each key at
  position ``first`` or later, the sum of exp(logit - lse) over the rows that see it and the query heads of its group:
  added to what it had, or set for the call's own tokens (all tokens where the call does not accumulate).
* evict: of each sequence and key head at most ``keep`` tokens stay: the ``first`` ones, the ``last`` ones and those of
  the others with the largest weights (of equal ones the earlier). K, V and weights move together, in order, to the
  sequence's first pages, or to those of ``to_table``. ``kept`` says where each came from.
"""

import math
import random

import torch

own = False

D = 128

# Head counts, clip lengths and context lengths are those of the benchmark's workloads (2, 24, 40 and 56 heads, 1152 to
# 67608 tokens), with grouped key heads where single tokens are served.
_LISTED = [
    # two answers to one prompt: the latency of a call
    dict(name="prefix, two sequences", op="prefix", kind="bf16", page=64, seqs=2, groups=1, hq=8, h=2, new=1, prefix=1152, lo=20, hi=77, mask="causal"),
    # a full decoding batch behind one long instruction
    dict(name="prefix, a batch", op="prefix", kind="bf16", page=64, seqs=64, groups=1, hq=40, h=8, new=1, prefix=33792, lo=64, hi=2048, mask="causal"),
    # the same over a quantised cache with several prefixes of uneven length and drafted tokens
    dict(name="prefix, groups", op="prefix", kind="e4m3", page=32, seqs=96, groups=5, hq=56, h=8, new=3, prefix=8704, lo=100, hi=4096, mask="causal"),
    # four continuations of one cached clip (h3: 9505 tokens, 56 heads), each attending both ways
    dict(name="prefix, continuations", op="prefix", kind="bf16", page=64, seqs=4, groups=1, hq=56, h=56, new=264, prefix=9505, lo=264, hi=264, mask="all"),
    # one user's decoding step
    dict(name="weigh, one sequence", op="weigh", kind="bf16", page=64, seqs=1, hq=8, h=2, new=1, lo=1152, hi=1152, mask="causal", window=0, first=4, add=True),
    # a decoding batch of ragged contexts
    dict(name="weigh, a batch", op="weigh", kind="bf16", page=64, seqs=64, hq=40, h=8, new=1, lo=512, hi=33792, mask="causal", window=0, first=4, add=True),
    # drafted tokens over a quantised cache, with a sliding window
    dict(name="weigh, few tokens", op="weigh", kind="e4m3", page=32, seqs=32, hq=24, h=8, new=4, lo=300, hi=8704, mask="causal", window=4096, first=0, add=True),
    # a long prompt taken in chunks
    dict(name="weigh, a chunk", op="weigh", kind="bf16", page=64, seqs=1, hq=40, h=8, new=2048, lo=33792, hi=33792, mask="causal", window=0, first=4, add=True),
    # the last rows of several prompts decide which of their tokens stay
    dict(name="weigh, observation rows", op="weigh", kind="e4m3", page=64, seqs=8, hq=24, h=24, new=64, lo=1152, hi=8704, mask="causal", window=0, first=4, add=False),
    # one user's cache is cut back by a block's worth
    dict(name="evict, one sequence", op="evict", kind="bf16", page=64, seqs=1, h=2, lo=1152, hi=1152, keep=1024, first=4, last=64, to=False),
    # a batch over its budget, some sequences still within it; to pages taken for it
    dict(name="evict, a batch", op="evict", kind="e4m3", page=32, seqs=64, h=8, lo=1024, hi=8704, keep=2048, first=4, last=256, to=True),
    # a long context at once, in its own pages (64k: 67608 tokens, 24 heads)
    dict(name="evict, a long context", op="evict", kind="bf16", page=64, seqs=1, h=24, lo=67608, hi=67608, keep=16384, first=64, last=1024, to=False),
]


def listed():
    return [dict(c) for c in _LISTED]


def _spread(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def _lengths(case):
    """(tokens of each sequence, its new rows, groups' first sequences, groups' prefixes): a plain function of the case."""
    rng = random.Random(1009 * case["seqs"] + 31 * case.get("new", 0) + case["lo"] + 7 * case["hi"])
    n = case["seqs"]
    lens = [case["hi"]] + [_spread(rng, case["lo"], case["hi"]) for _ in range(n - 1)]
    new = case.get("new", 0)
    news = [min(a, b) for a, b in zip([new] + [_spread(rng, 1, new) for _ in range(n - 1)], lens)] if new else []
    if case["op"] != "prefix":
        return lens, news, [], []
    starts = [0] + sorted(rng.sample(range(1, n), case["groups"] - 1)) + [n]
    prefixes = [case["prefix"]] + [rng.choice([0, 1, 2]) and _spread(rng, max(1, case["prefix"] // 32), case["prefix"])
                                   for _ in starts[2:]]
    of = [p for g, p in enumerate(prefixes) for _ in range(starts[g + 1] - starts[g])]
    return [a + p for a, p in zip(lens, of)], news, starts, prefixes


def _spans(case):
    """(row-key pairs, keys read, keys written) of one head, over all sequences."""
    lens, news, starts, prefixes = _lengths(case)
    pairs = keys = 0
    first, window = case.get("first", 0), case.get("window", 0)
    for n, m in zip(lens, news):
        if case["mask"] == "all":
            pairs, keys = pairs + m * max(0, n - first), keys + max(0, n - first)
            continue
        lo = [max(first, p + 1 - (window or n)) for p in range(n - m, n)]
        pairs += sum(max(0, p + 1 - x) for p, x in zip(range(n - m, n), lo))
        keys += max(0, n - lo[0])
    for g, p in enumerate(prefixes):  # read once
        shared = p // case["page"] * case["page"]
        keys -= shared * (starts[g + 1] - starts[g] - 1)
    return pairs, keys


def work(case):
    lens, news, _, _ = _lengths(case)
    cached = 2 * D if case["kind"] == "bf16" else D + 1  # bytes of a cached row
    h = case["h"]
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) - (0 if case["to"] else min(n, case["first"])) for n in lens if case["to"] or n > case["keep"])
        seen = sum(n for n in lens if n > case["keep"])
        return {"bytes": h * (4 * seen + kept * (4 * cached + 8) + 4 * len(lens) * case["keep"]), "flops": 0}
    rows, hq = sum(news), case["hq"]
    pairs, keys = _spans(case)
    if case["op"] == "weigh":
        return {"bytes": keys * h * (cached + (8 if case["add"] else 4)) + rows * hq * (2 * D + 4), "flops": 2 * D * hq * pairs}
    return {"bytes": 2 * keys * h * cached + rows * hq * (4 * D + 4), "flops": 4 * D * hq * pairs}


def draw(rng):
    while True:
        op = rng.choice(["prefix", "weigh", "evict"])
        h = rng.choice([1, 2, 8, 8, 24, 40])
        c = dict(op=op, kind=rng.choice(["bf16", "e4m3"]), page=rng.choice([16, 32, 64, 128]), seqs=_spread(rng, 1, 96), h=h)
        c["hi"] = _spread(rng, 40, 33792 if op != "prefix" else 4096)
        c["lo"] = _spread(rng, 1, c["hi"])
        if op == "evict":
            c.update(keep=_spread(rng, 16, c["hi"]), to=rng.random() < 0.5)
            c["first"], c["last"] = rng.randrange(c["keep"] // 4 + 1), rng.randrange(c["keep"] // 2 + 1)
        else:
            c["hq"] = h * rng.choice([1, 1, 3, 4, 5, 7, 8])
            c["mask"] = rng.choice(["causal", "causal", "all"])
            c["new"] = rng.choice([1, _spread(rng, 2, 8), _spread(rng, 9, 2048)])
            if op == "prefix":
                c.update(groups=min(c["seqs"], rng.choice([1, 1, 2, 3, 7])), prefix=_spread(rng, 100, 33792))
            else:
                c["window"] = _spread(rng, 16, 8192) if c["mask"] == "causal" and rng.random() < 0.3 else 0
                c.update(first=rng.choice([0, 4, 64]), add=rng.random() < 0.7)
            lens, news, _, _ = _lengths(c)
            # the plain form pads every sequence to the longest
            if c["hq"] > 64 or c["seqs"] * max(news) * c["hq"] * max(lens) > 2e9 or c["seqs"] * max(lens) * h > 1.8e7:
                continue
        w = work(c)
        if 2e5 <= w["bytes"] <= 8e8 and w["flops"] <= 6.8e11 and sum(_lengths(c)[0]) * h <= 1.5e7:
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


def _bytes(pages):
    """Codes as bytes, which indexing moves."""
    return pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(dev).manual_seed(seed)
    lens, news, starts, prefixes = _lengths(case)
    h, ps, bf, op = case["h"], case["page"], torch.bfloat16, case["op"]

    def normal(*shape, dtype=bf):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    # the pages of each sequence; whole pages of a prefix are those of its group's first sequence
    need, own_from = [-(-n // ps) for n in lens], [0] * len(lens)
    for k, p in enumerate(prefixes):
        for s in range(starts[k] + 1, starts[k + 1]):
            own_from[s] = p // ps
    more = -(-case["keep"] // ps) if op == "evict" and case["to"] else 0
    total = sum(need) - sum(own_from) + more * len(lens) + 3  # a few pages of the pool are free
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        mine = n - own_from[s]
        if own_from[s]:
            table[s, :own_from[s]] = table[max(x for x in starts if x <= s), :own_from[s]]
        table[s, own_from[s]:n] = order[at:at + mine]
        at += mine
    row_start = [0]
    for m in news:
        row_start.append(row_start[-1] + m)
    rows = row_start[-1]
    st = dict(op=op, page=ps, table=table, kv_len=i32(lens), k_exp=None, v_exp=None)
    # keys around a mean of their head, values of uneven size from token to token
    kv = [normal(total, h, ps, D) + normal(h, 1, D), normal(total, h, ps, D) * torch.exp(normal(total, 1, ps, 1))]
    for k, p in enumerate(prefixes):  # a prefix that ends inside a page: each sequence has a copy of that page's tokens
        if p % ps:
            pages = table[starts[k]:starts[k + 1], p // ps].long()
            for x in kv:
                x[pages, :, :p % ps] = x[pages[:1], :, :p % ps]
    if case["kind"] == "e4m3":
        kv[0], st["k_exp"] = _quantise(kv[0])
        kv[1], st["v_exp"] = _quantise(kv[1])
    st["k_pages"], st["v_pages"] = kv
    if op != "prefix":
        # weights so far: uneven, and nothing at all on many keys
        w = torch.exp(2 * normal(total, h, ps, dtype=torch.float32) - 6)
        st["weights"] = torch.where(normal(total, h, ps, dtype=torch.float32) > 0.5, 0.0, w)
        st["first"] = case["first"]
    if op == "evict":
        st.update(keep=case["keep"], last=case["last"], to_table=None)
        if case["to"]:
            st["to_table"] = order[at:at + more * len(lens)].view(len(lens), more).clone()
        st["kept"] = torch.full((len(lens), h, case["keep"]), -1, dtype=torch.int32, device=dev)
        st["new_len"] = torch.zeros_like(st["kv_len"])
        return st
    # q is a strided part of the projection's output
    st["q"] = (2.0 * normal(rows, case["hq"] + 2 * h, D))[:, :case["hq"]]
    st.update(rows=rows, new=max(news), row_start=i32(row_start), causal=case["mask"] == "causal", window=case.get("window", 0))
    if op == "prefix":
        st.update(group_start=i32(starts), prefix_len=i32(prefixes))
        st["o"] = torch.zeros((rows, case["hq"], D), dtype=bf, device=dev)
        st["lse"] = torch.zeros((rows, case["hq"]), dtype=torch.float32, device=dev)
        return st
    st["add"] = case["add"]
    x, s, i = _logits(st)
    st["lse"] = _packed(torch.logsumexp(x, -1, keepdim=True), st, s, i).squeeze(-1).contiguous()
    return st


def _rows(st):
    """Sequence, place in it and position of every row."""
    r = torch.arange(st["rows"], device=st["table"].device)
    s = torch.searchsorted(st["row_start"][1:], r, right=True)
    n = st["row_start"][1:] - st["row_start"][:-1]
    return s, r - st["row_start"][s], (st["kv_len"] - n)[s] + r - st["row_start"][s]


def _padded_cache(pages, exp, table):
    """[sequences, heads, tokens, 128] of every sequence's pages, in 32 bits."""
    t = table.long()
    x = _bytes(pages)[t].view(pages.dtype).float()
    if exp is not None:
        x *= _two(exp[t].int().unsqueeze(-1) - 127)
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _padded_rows(x, st, s, i):
    """Rows [rows, Hq, n] as [sequences, heads, new tokens x group, n], zeros where there is none."""
    hq, h = x.shape[1], st["k_pages"].shape[1]
    y = torch.zeros((st["table"].shape[0], st["new"], hq, x.shape[2]), dtype=torch.float32, device=x.device)
    y[s, i] = x.float()
    return y.unflatten(2, (h, hq // h)).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _packed(y, st, s, i):
    """The inverse of _padded_rows."""
    hq, h = st["q"].shape[1], st["k_pages"].shape[1]
    return y.unflatten(2, (st["new"], hq // h)).permute(0, 2, 1, 3, 4).flatten(2, 3)[s, i]


def _logits(st):
    """Logits [sequences, heads, new tokens x group, tokens], -inf where a row does not see a key."""
    q, kv_len = st["q"], st["kv_len"]
    s, i, pos = _rows(st)
    group = q.shape[1] // st["k_pages"].shape[1]
    x = _padded_rows(q, st, s, i) @ _padded_cache(st["k_pages"], st["k_exp"], st["table"]).transpose(-1, -2)
    x *= 1.0 / math.sqrt(D)
    at = torch.full((kv_len.shape[0], st["new"]), -1, dtype=torch.int64, device=q.device)
    at[s, i] = pos
    at = at[..., None]
    j = torch.arange(x.shape[3], device=q.device)
    seen = (j < kv_len[:, None, None]) & (at >= 0)
    if st["causal"]:
        seen = seen & (j <= at)
    if st["window"]:
        seen = seen & (j > at - st["window"])
    x.masked_fill_(~seen.unsqueeze(1).unsqueeze(3).expand(-1, x.shape[1], -1, group, -1).flatten(2, 3), -math.inf)
    return x, s, i


def _plain_prefix(st):
    x, s, i = _logits(st)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = x @ _padded_cache(st["v_pages"], st["v_exp"], st["table"])
    o = torch.where(total > 0, o / total, 0.0)
    return _packed(o, st, s, i).to(st["q"].dtype), _packed(top + total.log(), st, s, i).squeeze(-1)


def _plain_weigh(st):
    x, s, i = _logits(st)
    received = x.sub_(_padded_rows(st["lse"].unsqueeze(-1), st, s, i)).exp_().sum(2)  # [sequences, heads, tokens]
    table, kv_len, ps = st["table"].long(), st["kv_len"][:, None], st["page"]
    j = torch.arange(received.shape[2], device=table.device)
    page, slot = table[:, j // ps], (j % ps).expand(table.shape[0], -1)
    before = st["weights"][page, :, slot].transpose(1, 2)
    news = (st["row_start"][1:] - st["row_start"][:-1])[:, None]
    old = (j < kv_len - news) if st["add"] else torch.zeros_like(j < kv_len)
    after = torch.where(old.unsqueeze(1), before, 0.0) + received
    # places without a token go to a page of their own
    free = st["weights"].shape[0]
    page = torch.where((j < kv_len) & (j >= st["first"]), page, free)
    w = torch.cat([st["weights"], torch.zeros_like(st["weights"][:1])])
    w[page, :, slot] = after.transpose(1, 2)
    st["weights"].copy_(w[:free])
    return st["weights"]


def _plain_evict(st):
    table, kv_len, ps, keep = st["table"].long(), st["kv_len"].long(), st["page"], st["keep"]
    to = table if st["to_table"] is None else st["to_table"].long()
    n, h = table.shape[0], st["k_pages"].shape[1]
    w = st["weights"][table].permute(0, 2, 1, 3).flatten(2)  # [sequences, heads, tokens]
    if w.shape[2] < keep:
        w = torch.nn.functional.pad(w, (0, keep - w.shape[2]))
    j = torch.arange(w.shape[2], device=w.device)
    n_of = kv_len[:, None, None]
    w = torch.where((j < st["first"]) | (j >= n_of - st["last"]), math.inf, w)
    w = torch.where(j < n_of, w, -math.inf)
    kept = torch.sort(w, dim=2, descending=True, stable=True).indices[..., :keep].sort(2).values
    there = kept < n_of
    # where a sequence has fewer tokens, its first one is moved again
    src, dst = torch.where(there, kept, 0), torch.where(there, torch.arange(keep, device=w.device), 0)
    s, head = torch.arange(n, device=w.device)[:, None, None], torch.arange(h, device=w.device)[None, :, None]
    from_page, to_page = table[s, src // ps], to[s, dst // ps]
    outs = [st["k_pages"], st["v_pages"], st["weights"]] + ([st["k_exp"], st["v_exp"]] if st["k_exp"] is not None else [])
    for x in map(_bytes, outs):
        x[to_page, head, dst % ps] = x[from_page, head, src % ps]
    return (*outs, torch.where(there, kept, -1).int(), kv_len.clamp(max=keep).int())


def run(state):
    st = state
    if own:
        import block_sparse_routed_gb300 as bsr

        if st["op"] == "prefix":
            if "ws" not in st:  # a server keeps one workspace
                st["ws"] = bsr.prefix_workspace(st["q"], st["k_pages"], st["table"], st["group_start"], max_new=st["new"])
            return bsr.prefix_attn(st["q"], st["k_pages"], st["v_pages"], st["table"], st["row_start"], st["kv_len"],
                                   st["group_start"], st["prefix_len"], max_new=st["new"], causal=st["causal"],
                                   k_exp=st["k_exp"], v_exp=st["v_exp"], o=st["o"], lse=st["lse"], ws=st["ws"])
        if st["op"] == "weigh":
            return bsr.cache_weigh(st["q"], st["lse"], st["weights"], st["k_pages"], st["table"], st["row_start"], st["kv_len"],
                                   max_new=st["new"], causal=st["causal"], window=st["window"], first=st["first"],
                                   accumulate=st["add"], k_exp=st["k_exp"])
        bsr.cache_evict(st["k_pages"], st["v_pages"], st["weights"], st["table"], st["kv_len"], st["keep"], first=st["first"],
                        last=st["last"], to_table=st["to_table"], k_exp=st["k_exp"], v_exp=st["v_exp"], kept=st["kept"],
                        new_len=st["new_len"])
        exps = (st["k_exp"], st["v_exp"]) if st["k_exp"] is not None else ()
        return (st["k_pages"], st["v_pages"], st["weights"], *exps, st["kept"], st["new_len"])
    return {"prefix": _plain_prefix, "weigh": _plain_weigh, "evict": _plain_evict}[st["op"]](st)


def _exact_pages(pages, exp):
    """Cached rows [n, H, page_size, 128] in 64 bits."""
    if exp is None:
        return pages.double()
    code = pages.view(torch.uint8).int()
    m, e = (code & 7).double(), (code >> 3) & 15
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(code >= 128, -mag, mag) * torch.exp2(exp.double() - 127).unsqueeze(-1)


def _exact_rows(st, name, s, n):
    """The first n cached rows of a sequence [H, n, 128] in 64 bits."""
    t = st["table"][s, :-(-n // st["page"])].long()
    exp = st[name[0] + "_exp"]
    x = _exact_pages(_bytes(st[name])[t].view(st[name].dtype), None if exp is None else exp[t])
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def exact(case, seed):
    st = prepare(case, seed)
    lens, news, _, _ = _lengths(case)
    ps, table, dev = case["page"], st["table"].long(), st["table"].device
    if case["op"] == "evict":
        names = ["k_pages", "v_pages", "weights"] + (["k_exp", "v_exp"] if st["k_exp"] is not None else [])
        value = {x: st[x] if "exp" in x else _exact_pages(st[x], None) if "pages" in x and st["k_exp"] is not None else st[x].double() for x in names}
        new = {x: value[x].clone() for x in names}
        to = table if st["to_table"] is None else st["to_table"].long()
        heads = torch.arange(case["h"], device=dev)[:, None]
        for s, n in enumerate(lens):
            stay = min(n, case["keep"])
            j = torch.arange(n, device=dev)
            w = st["weights"][table[s, j // ps], :, j % ps].double().T  # [H, n]
            always = (j < case["first"]) | (j >= n - case["last"]) if n > case["keep"] else j >= 0
            rank = torch.argsort(torch.where(always, -math.inf, -w), dim=1, stable=True)
            chosen = torch.zeros_like(w, dtype=torch.bool).scatter_(1, rank[:, :stay], True)
            k = torch.nonzero(chosen)[:, 1].view(case["h"], stay)
            i = torch.arange(stay, device=dev)
            for x in names:
                new[x][to[s, i // ps], heads, i % ps] = value[x][table[s, k // ps], heads, k % ps]
            st["kept"][s, :, :stay] = k.int()
            st["new_len"][s] = stay
        return (*(new[x] for x in names), st["kept"], st["new_len"])
    outs, r0 = [], 0
    weights = st["weights"].double() if case["op"] == "weigh" else None
    for s, (n, m) in enumerate(zip(lens, news)):
        k = _exact_rows(st, "k_pages", s, n)
        v = _exact_rows(st, "v_pages", s, n) if weights is None else None
        q = st["q"][r0:r0 + m].double()
        lse_in = st["lse"][r0:r0 + m].double()
        r0 += m
        j = torch.arange(n, device=dev)
        p = torch.arange(n - m, n, device=dev)[:, None]
        hidden = torch.zeros((m, n), dtype=torch.bool, device=dev)
        if case["mask"] == "causal":
            hidden = j[None] > p
            if case.get("window"):
                hidden |= j[None] <= p - case["window"]
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=dev)
        got = torch.zeros((case["h"], n), dtype=torch.float64, device=dev)
        for head in range(case["hq"]):
            kh = head // (case["hq"] // case["h"])
            x = torch.mm(q[:, head], k[kh].T) / math.sqrt(D)
            x[hidden] = -math.inf
            if weights is None:
                lse[:, head] = torch.logsumexp(x, 1)
                o[:, head] = torch.mm(torch.exp(x - lse[:, head, None]), v[kh])
            else:
                got[kh] += torch.exp(x - lse_in[:, head, None]).sum(0)
        if weights is None:
            outs.append((o, lse))
            continue
        f = case["first"]
        page, slot = table[s, j // ps][f:], (j % ps)[f:]
        had = weights[page, :, slot]
        had[(max(0, n - m - f) if case["add"] else 0):] = 0
        weights[page, :, slot] = had + got[:, f:].T
    return weights if weights is not None else tuple(torch.cat(x) for x in zip(*outs))
