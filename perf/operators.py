"""The windowed attention, the attention of one new position over a paged cache, and the
page operations of that cache: the cases they are measured on, in a plain form and as the
library's calls.

Three operators, by a case's "op":

* ``window``: attention in which key j is visible to position p of a clip of n positions
  iff j < n, j <= p + right and (j >= p - left or j < sinks); a negative left or right is
  no limit. Rows at or past n are left as they were.
* ``paged``: the same for the one newest position of each sequence (p = n - 1), its keys
  and values in pages that a table names; a sequence of length 0 gives zeros.
* ``pages``: the cache's own operations. "branch" forks sequences and makes every one a
  position longer, which copies the partly filled pages they share; "retire" frees some
  sequences and compacts what is left; "append" writes new keys and values into pages.
"""
import math

import torch

own = False

PAGE_KINDS = ("branch", "retire", "append")


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # One 30-second clip (374 positions, ten heads of 128) with 50 positions of context
        # on each side: the smallest call of a local encoder, where latency counts.
        dict(name="window_30s", op="window", batch=1, T=374, heads=10, kv_heads=10, head_dim=128, left=50, right=50,
             sinks=0, ragged=False),
        # Sixteen one-minute clips of different lengths in one padded batch, causal with
        # half a minute of history and the first four positions kept.
        dict(name="window_16x60s", op="window", batch=16, T=749, heads=10, kv_heads=10, head_dim=128, left=375, right=0,
             sinks=4, ragged=True),
        # One hour, causal: a minute of history and eight first positions.
        dict(name="window_1h", op="window", batch=1, T=44999, heads=10, kv_heads=10, head_dim=128, left=750, right=0,
             sinks=8, ragged=False),
        # The heads of the timestamp adapter (16 of 64) over half an hour on its 40 ms grid,
        # ten seconds to each side.
        dict(name="window_hd64", op="window", batch=1, T=44998, heads=16, kv_heads=16, head_dim=64, left=250, right=250,
             sinks=0, ragged=False),
        # A long prompt with grouped heads: 32 query heads share two key heads.
        dict(name="window_grouped", op="window", batch=2, T=8191, heads=32, kv_heads=2, head_dim=128, left=1023, right=0,
             sinks=4, ragged=True),
        # One live stream, a minute of cache.
        dict(name="paged_one", op="paged", batch=1, length=750, ragged=False, heads=10, kv_heads=10, head_dim=128,
             page=16, left=-1, sinks=0),
        # 64 live streams that are an hour old: each new position sees a minute and eight
        # first positions of its 45,000.
        dict(name="paged_live", op="paged", batch=64, length=45000, ragged=True, heads=10, kv_heads=10, head_dim=128,
             page=16, left=749, sinks=8),
        # A few hour-long sequences with grouped heads, the whole cache visible: few rows,
        # a long axis.
        dict(name="paged_long", op="paged", batch=3, length=45000, ragged=True, heads=32, kv_heads=2, head_dim=128,
             page=64, left=-1, sinks=0),
        # A full batch of uneven lengths: the most bytes.
        dict(name="paged_batch", op="paged", batch=64, length=8190, ragged=True, heads=10, kv_heads=10, head_dim=128,
             page=16, left=-1, sinks=0),
        # Eight streams, each continued by four hypotheses from a two-layer cache: small.
        dict(name="pages_branch", op="pages", kind="branch", layers=2, kv_heads=10, head_dim=128, page=16, sequences=32,
             length=375, every=4),
        # Half of 96 streams of a 32-layer cache end; the rest move together.
        dict(name="pages_retire", op="pages", kind="retire", layers=32, kv_heads=10, head_dim=128, page=16,
             sequences=96, length=250, every=2),
        # The keys and values of sixteen prompts of up to a minute written to their pages.
        dict(name="pages_append", op="pages", kind="append", layers=1, kv_heads=10, head_dim=128, page=16,
             sequences=16, length=749, every=1),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _heads(rng):
    return rng.choice([(10, 10, 128), (16, 16, 64), (32, 2, 128), (8, 4, 128), (12, 4, 64), (10, 2, 128)])


def _draw(rng):
    op = rng.choice(["window", "paged", "pages"])
    heads, kv_heads, head_dim = _heads(rng)
    if op == "window":
        T = _log(rng, 1, 45000)
        return dict(op=op, batch=_log(rng, 1, 16), T=T, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                    left=rng.choice([-1, 0, _log(rng, 1, 2000)]), right=rng.choice([0, 0, -1, _log(rng, 1, 500)]),
                    sinks=rng.choice([0, 1, _log(rng, 2, 64)]), ragged=rng.random() < 0.5)
    if op == "paged":
        return dict(op=op, batch=_log(rng, 1, 256), length=_log(rng, 1, 45000), ragged=rng.random() < 0.7, heads=heads,
                    kv_heads=kv_heads, head_dim=head_dim, page=rng.choice([8, 16, 32, 64, 128]),
                    left=rng.choice([-1, -1, _log(rng, 1, 4000)]), sinks=rng.choice([0, _log(rng, 1, 64)]))
    return dict(op=op, kind=rng.choice(PAGE_KINDS), layers=rng.choice([1, 2, 8, 32]), kv_heads=kv_heads,
                head_dim=head_dim, page=rng.choice([8, 16, 32, 64]), sequences=_log(rng, 2, 128),
                length=_log(rng, 1, 4000), every=rng.choice([2, 3, 4]))


def _footprint(c):
    """Bytes that the case's state, or the plain form's largest temporary, takes."""
    if c["op"] == "window":
        span, _ = _span(c)
        block = _block(c)
        return 4 * c["batch"] * c["heads"] * -(-c["T"] // block) * block * (min(span + block, c["T"]) + c["sinks"])
    if c["op"] == "paged":
        return 4 * _pool_pages(c) * c["page"] * c["kv_heads"] * c["head_dim"]
    return 4 * c["layers"] * _pool_pages(c) * c["page"] * c["kv_heads"] * c["head_dim"]


def draw(rng):
    """One more case of these ranges, no dearer than the largest listed one of its operator."""
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0, "flops": 0, "room": 0})
        m.update(bytes=max(m["bytes"], w["bytes"]), flops=max(m["flops"], w["flops"]),
                 room=max(m["room"], _footprint(c)))
    while True:
        c = _draw(rng)
        w, m = work(c), most[c["op"]]
        if w["bytes"] <= m["bytes"] and w["flops"] <= max(m["flops"], 1) and _footprint(c) <= m["room"]:
            return c


def _lengths(n, top, ragged):
    """Lengths of n sequences: all `top`, or spread over [top / 4, top] with one at each end."""
    if not ragged:
        return [top] * n
    low = top - top * 3 // 4
    got = [low + int((top - low + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]
    got[-1] = top
    return got


def _span(c):
    """(left + right, both), each capped to the clip."""
    left = c["T"] if c["left"] < 0 else min(c["left"], c["T"])
    right = c["T"] if c["right"] < 0 else min(c["right"], c["T"])
    return left + right, (left, right)


def _block(c):
    """Queries that the plain form takes at a time."""
    return max(64, min(512, c["T"]))


def _pool_pages(c):
    """Pages of the case's pool: those in use and some free ones."""
    if c["op"] == "paged":
        used = sum(-(-n // c["page"]) for n in _lengths(c["batch"], c["length"], c["ragged"]))
        return used + 7
    used = sum(-(-n // c["page"]) for n in _lengths(c["sequences"], c["length"], True))
    return used + 2 * c["sequences"] + 5


def _ceil(n, page):
    return -(-n // page)


# --------------------------------------------------------------------------- work

def _visible_pairs(n, left, right, sinks):
    """Visible (position, key) pairs of one clip of n positions."""
    left = n if left < 0 else min(left, n)
    right = n if right < 0 else min(right, n)
    p = torch.arange(n, dtype=torch.int64)
    hi = torch.clamp(p + right, max=n - 1)
    lo = torch.clamp(p - left, min=0)
    window = int((hi - lo + 1).sum())
    extra = torch.minimum(torch.minimum(torch.full_like(p, sinks), lo), hi + 1)
    return window + int(torch.clamp(extra, min=0).sum())


def work(case):
    c = case
    if c["op"] == "window":
        lens = _lengths(c["batch"], c["T"], c["ragged"])
        rows = sum(lens)
        pairs = sum(_visible_pairs(n, c["left"], c["right"], c["sinks"]) for n in lens)
        d = c["head_dim"]
        return {"bytes": 2 * d * rows * (2 * c["heads"] + 2 * c["kv_heads"]), "flops": 4 * d * c["heads"] * pairs}
    if c["op"] == "paged":
        keys = 0
        for n in _lengths(c["batch"], c["length"], c["ragged"]):
            window = n if c["left"] < 0 else min(n, c["left"] + 1)
            keys += window + min(c["sinks"], n - window)
        d = c["head_dim"]
        return {"bytes": 4 * d * (c["kv_heads"] * keys + c["heads"] * c["batch"]) + 4 * keys // c["page"],
                "flops": 4 * d * c["heads"] * keys}
    plan = _Plan(c)
    page_bytes = 4 * c["layers"] * c["kv_heads"] * c["page"] * c["head_dim"]
    table_bytes = 8 * plan.sequences * plan.max_pages
    if c["kind"] == "append":
        return {"bytes": 8 * sum(plan.lengths) * c["kv_heads"] * c["head_dim"], "flops": 0}
    if c["kind"] == "branch":
        # the partly filled last page of every group of two or more is copied for each of them
        copies = sum(1 for i in range(plan.sequences) if plan.lengths[i - i % c["every"]] % c["page"] and
                     (i % c["every"] or i + 1 < plan.sequences))
        return {"bytes": 2 * copies * page_bytes + table_bytes, "flops": 0}
    live = sum(_ceil(n, c["page"]) for i, n in enumerate(plan.lengths) if i % c["every"])
    total = sum(_ceil(n, c["page"]) for n in plan.lengths)
    # pages are handed out at random, so a share live / pool of the tail has to move
    moved = live * (_pool_pages(c) - live) // _pool_pages(c) if total else 0
    return {"bytes": 2 * moved * page_bytes + table_bytes, "flops": 0}


class _Plan:
    """Sizes of a page case that follow from the case alone."""

    def __init__(self, c):
        self.sequences = c["sequences"]
        self.lengths = _lengths(self.sequences, c["length"], True)
        self.max_pages = _ceil(c["length"] + 1, c["page"]) + 1


# --------------------------------------------------------------------------- inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _unit(g, *shape):
    """Rows of RMS 1, as the encoder's normalised queries and keys are."""
    x = _randn(g, *shape)
    return x.mul_(shape[-1] ** 0.5 / torch.linalg.vector_norm(x, dim=-1, keepdim=True, dtype=torch.float32))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, lengths, max_pages, page, pool):
    """Page tables of sequences of these lengths: distinct pages in random order, -1 past the end."""
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    counts = _ints([_ceil(n, page) for n in lengths]).long()
    column = torch.arange(max_pages, device="cuda")
    at = (torch.cumsum(counts, 0) - counts)[:, None] + column
    return torch.where(column < counts[:, None], order[at.clamp(max=pool - 1)], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    c, g = case, _rng(seed)
    s = {"case": c}
    if c["op"] == "window":
        B, T, d = c["batch"], c["T"], c["head_dim"]
        s["q"], s["k"] = _unit(g, B, c["heads"], T, d), _unit(g, B, c["kv_heads"], T, d)
        s["v"] = _randn(g, B, c["kv_heads"], T, d)
        s["lengths"] = _ints(_lengths(B, T, True)) if c["ragged"] else None
        s["o"] = torch.zeros(B * T, c["heads"] * d, dtype=torch.bfloat16, device="cuda")
        return s
    if c["op"] == "paged":
        lengths = _lengths(c["batch"], c["length"], c["ragged"])
        pool, d = _pool_pages(c), c["head_dim"]
        max_pages = _ceil(c["length"], c["page"])
        s["table"], s["lengths"] = _table(g, lengths, max_pages, c["page"], pool), _ints(lengths)
        s["k"] = _unit(g, 1, pool, c["kv_heads"], c["page"], d)
        s["v"] = _randn(g, 1, pool, c["kv_heads"], c["page"], d)
        s["q"] = _unit(g, c["batch"], c["heads"], d)
        s["o"] = torch.zeros(c["batch"], c["heads"] * d, dtype=torch.bfloat16, device="cuda")
    else:
        plan = _Plan(c)
        n, pool, d = plan.sequences, _pool_pages(c), c["head_dim"]
        max_pages = plan.max_pages
        s["k"] = _randn(g, c["layers"], pool, c["kv_heads"], c["page"], d)
        s["v"] = _randn(g, c["layers"], pool, c["kv_heads"], c["page"], d)
        s["table"], s["lengths"] = _table(g, plan.lengths, max_pages, c["page"], pool), _ints(plan.lengths)
        if c["kind"] == "branch":
            # every sequence goes on from the first of its group
            s["src"], s["dst"] = _ints([i - i % c["every"] for i in range(n)]), _ints(list(range(n)))
            s["longer"] = _ints([plan.lengths[i - i % c["every"]] + 1 for i in range(n)])
        elif c["kind"] == "retire":
            s["ended"] = _ints([i for i in range(n) if i % c["every"] == 0])
            s["none"] = torch.zeros_like(s["ended"])
        else:
            T = c["length"]
            s["new_k"], s["new_v"] = _randn(g, n, c["kv_heads"], T, d), _randn(g, n, c["kv_heads"], T, d)
            s["starts"] = _ints([0] * n)
        # what the calls write their tables to: the ones above stay, so a pass can be run again
        s["tables"] = [torch.empty_like(s["table"]) for _ in range(2)]
        s["lens"] = [torch.empty_like(s["lengths"]) for _ in range(2)]
    if own:
        from speech_audio_encoder_b200 import api
        s["cache"] = api.PagedCache(s["k"], s["v"], s["table"], s["lengths"])
        if c["op"] == "pages":
            s["after"] = [api.PagedCache(s["k"], s["v"], t, n) for t, n in zip(s["tables"], s["lens"])]
        else:
            s["workspace"] = api.attention_paged_workspace(s["cache"], c["batch"], c["heads"])
    return s


# --------------------------------------------------------------------------- plain forms

def _plain_window(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    B, T, H, d = c["batch"], c["T"], c["heads"], c["head_dim"]
    share, (left, right), step, sinks = H // c["kv_heads"], _span(c)[1], _block(c), min(c["sinks"], c["T"])
    blocks = -(-T // step)
    left, right = min(left, blocks * step), min(right, blocks * step)
    if left + right + step >= 2 * T:  # the band is the whole clip: one block of all keys
        left, right, step, blocks = 0, 0, T, 1
        left_limit, right_limit = _span(c)[1]
    else:
        left_limit, right_limit = left, right
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, dtype=torch.int32, device=q.device)

    def banded(x):  # [B, kv, T, d] -> [B, kv, 1, blocks, d, keys of the block]
        x = torch.nn.functional.pad(x.float(), (0, 0, left, blocks * step - T + right))
        return x.unfold(2, step + left + right, step)[:, :, None]

    qf = torch.nn.functional.pad(q.float(), (0, 0, 0, blocks * step - T))
    qf = qf.reshape(B, c["kv_heads"], share, blocks, step, d)
    p = torch.arange(blocks * step, device=q.device).reshape(blocks, step, 1)
    j = torch.arange(step + left + right, device=q.device) - left + step * torch.arange(blocks, device=q.device)[:, None, None]
    n = lengths.long().reshape(B, 1, 1, 1)
    seen = (j >= 0) & (j < n) & (j <= p + right_limit) & ((j >= p - left_limit) | (j < sinks))
    scores = qf @ banded(k) / math.sqrt(d)
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    if sinks and left_limit < T:
        ks, vs = (x[:, :, :sinks].float().reshape(B, c["kv_heads"], 1, 1, sinks, d) for x in (k, v))
        i = torch.arange(sinks, device=q.device)
        # those of the first keys that the band above has not got
        far = (i < n) & (i <= p + right_limit) & (i < p - left_limit) & (i < p // step * step - left)
        more = (qf @ ks.transpose(-1, -2) / math.sqrt(d)).masked_fill(~far[:, None, None], float("-inf"))
        scores = torch.cat([scores, more], -1)
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    del scores
    total = weights.sum(-1, keepdim=True)
    out = weights[..., :step + left + right] @ banded(v).transpose(-1, -2)
    if sinks and left_limit < T:
        out = out + weights[..., step + left + right:] @ vs
    out = (out / total).reshape(B, H, blocks * step, d)[:, :, :T].transpose(1, 2).reshape(B * T, H * d)
    row = (torch.arange(T, device=q.device) < lengths[:, None]).reshape(B * T, 1)
    s["o"].copy_(torch.where(row, out, s["o"].float()))
    return s["o"]


def _plain_paged(s):
    c, d = s["case"], s["case"]["head_dim"]
    n = s["lengths"].long()[:, None]
    top = s["table"].shape[1] * c["page"]
    window = top if c["left"] < 0 else min(top, c["left"] + 1)
    sinks = min(c["sinks"], top - window)
    # positions of the keys: the window, which ends at the newest, then the first ones before it
    j = n - 1 - torch.arange(window, device=n.device)
    first = torch.arange(sinks, device=n.device).expand(n.shape[0], sinks)
    j = torch.cat([j, torch.where(first < n - window, first, -1)], 1)
    page = torch.gather(s["table"].long(), 1, (j // c["page"]).clamp(0, s["table"].shape[1] - 1))
    seen = (j >= 0) & (page >= 0)
    at = page.clamp(min=0), j.clamp(min=0) % c["page"]
    k = s["k"][0][at[0], :, at[1]].float()  # [batch, keys, kv_heads, d]
    q = s["q"].float().reshape(c["batch"], c["kv_heads"], -1, d)
    scores = torch.einsum("bhgd,bnhd->bhgn", q, k) / math.sqrt(d)
    del k
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    high = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(high == float("-inf"), 0.0, high))
    weights = weights / weights.sum(-1, keepdim=True).clamp(min=1e-30)
    v = s["v"][0][at[0], :, at[1]].float()
    out = torch.einsum("bhgn,bnhd->bhgd", weights, v)
    s["o"].copy_(out.reshape(c["batch"], -1))
    return s["o"]


def _references(table, lengths, page, pool):
    """How many used entries name each page, and which entries are used."""
    used = torch.arange(table.shape[1], device=table.device) < -(-lengths.long() // page)[:, None]
    used = used & (table >= 0)
    return torch.bincount(torch.where(used, table, pool).long().reshape(-1), minlength=pool + 1)[:pool], used


def _plain_resize(s, table, lengths, rows, new):
    """Tables and lengths after the rows have got their new lengths; pages copied on the way."""
    page, pool = s["case"]["page"], s["k"].shape[1]
    table, lengths, old = table.clone(), lengths.clone(), lengths[rows.long()].long()
    rows, new, column = rows.long(), new.long(), torch.arange(table.shape[1], device=table.device)
    kept = torch.minimum(old, new)
    lengths[rows] = kept.int()
    table[rows] = torch.where(column < -(-kept // page)[:, None], table[rows], -1)
    count, _ = _references(table, lengths, page, pool)
    last = (kept // page)[:, None]
    name = torch.gather(table[rows], 1, last.clamp(max=table.shape[1] - 1)).long()
    shared = (count[name.clamp(min=0)] > 1) & (name >= 0) & (kept % page > 0)[:, None] & (new > kept)[:, None]
    fresh = (column >= -(-kept // page)[:, None]) & (column < -(-new // page)[:, None])
    need = fresh | (shared & (column == last))
    got = torch.nonzero(count == 0)[:, 0][:int(need.sum())]
    row = table[rows]
    row[need] = got.int()
    source, target = name[shared], torch.gather(row, 1, last.clamp(max=table.shape[1] - 1)).long()[shared]
    s["k"][:, target], s["v"][:, target] = s["k"][:, source], s["v"][:, source]
    table[rows] = row
    lengths[rows] = new.int()
    return table, lengths


def _plain_compact(s, table, lengths):
    page, pool = s["case"]["page"], s["k"].shape[1]
    count, used = _references(table, lengths, page, pool)
    live = count > 0
    index = torch.arange(pool, device=table.device)
    m = live.sum()
    source, target = torch.nonzero(live & (index >= m))[:, 0], torch.nonzero(~live & (index < m))[:, 0]
    s["k"][:, target], s["v"][:, target] = s["k"][:, source], s["v"][:, source]
    index[source] = target
    return torch.where(used, index[table.clamp(min=0).long()].int(), -1)


def _plain_pages(s):
    c = s["case"]
    if c["kind"] == "append":
        n, T = s["lengths"].long()[:, None], c["length"]
        position = s["starts"].long()[:, None] + torch.arange(T, device=n.device)
        at = torch.gather(s["table"].long(), 1, position // c["page"])
        row, token = torch.nonzero((position < n) & (at >= 0), as_tuple=True)
        page, slot = at[row, token], position[row, token] % c["page"]
        s["k"][0][page, :, slot], s["v"][0][page, :, slot] = s["new_k"][row, :, token], s["new_v"][row, :, token]
        return s["k"], s["v"]
    if c["kind"] == "branch":
        table, lengths = s["table"].clone(), s["lengths"].clone()
        table[s["dst"].long()], lengths[s["dst"].long()] = s["table"][s["src"].long()], s["lengths"][s["src"].long()]
        table, lengths = _plain_resize(s, table, lengths, s["dst"], s["longer"])
    else:
        table, lengths = _plain_resize(s, s["table"], s["lengths"], s["ended"], s["none"])
        table = _plain_compact(s, table, lengths)
    return s["k"], s["v"], table, lengths


# --------------------------------------------------------------------------- one pass

def _own(s):
    from speech_audio_encoder_b200 import api
    c = s["case"]
    if c["op"] == "window":
        return api.sal_attention_window(s["q"], s["k"], s["v"], left=c["left"], right=c["right"], sinks=c["sinks"],
                                        lengths=s["lengths"], out=s["o"])
    cache = s["cache"]
    if c["op"] == "paged":
        return api.sal_attention_paged(s["q"], cache, left=c["left"], sinks=c["sinks"], out=s["o"],
                                       workspace=s["workspace"])
    if c["kind"] == "append":
        api.sal_cache_append(cache, s["new_k"], s["new_v"], s["starts"])
        return cache.k, cache.v
    first, second = s["after"]
    if c["kind"] == "branch":
        api.sal_cache_fork(cache, s["src"], s["dst"], out=first)
        api.sal_cache_resize(first, s["dst"], s["longer"], out=second)
    else:
        api.sal_cache_resize(cache, s["ended"], s["none"], out=first)
        api.sal_cache_compact(first, out=second)
    return second.k, second.v, second.table, second.lengths


def run(state):
    if own:
        return _own(state)
    return {"window": _plain_window, "paged": _plain_paged, "pages": _plain_pages}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- in 64 bits

def _softmax_rows(q, k, v, seen):
    """softmax(q k^T / sqrt(d)) v over the keys that `seen` allows, in 64 bits."""
    scores = (q @ k.T) * (q.shape[-1] ** -0.5)
    scores[~seen] = -math.inf
    return torch.softmax(scores, -1) @ v


def exact(case, seed):
    c = case
    if c["op"] == "pages":
        return None  # pages are moved, not computed
    s = prepare(c, seed)
    d, share = c["head_dim"], c["heads"] // c["kv_heads"]
    if c["op"] == "window":
        B, T = c["batch"], c["T"]
        if B * c["heads"] * -(-T // 1024) > 12000:
            return None
        out = torch.zeros(B, T, c["heads"], d, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(B, T, c["ragged"])):
            for p0 in range(0, n, 1024):
                p1 = min(n, p0 + 1024)
                low = 0 if c["left"] < 0 else max(0, p0 - c["left"])
                high = n if c["right"] < 0 else min(n, p1 + c["right"])
                early = min(c["sinks"], low)
                keys = torch.cat([torch.arange(early), torch.arange(low, high)]).cuda()
                at = torch.arange(p0, p1).cuda()[:, None]
                seen = torch.ones(p1 - p0, keys.numel(), dtype=torch.bool, device="cuda")
                if c["right"] >= 0:
                    seen &= keys <= at + c["right"]
                if c["left"] >= 0:
                    seen &= (keys >= at - c["left"]) | (keys < c["sinks"])
                for h in range(c["heads"]):
                    out[b, p0:p1, h] = _softmax_rows(s["q"][b, h, p0:p1].double(), s["k"][b, h // share][keys].double(),
                                                     s["v"][b, h // share][keys].double(), seen)
        return out.reshape(B * T, -1)
    out = torch.zeros(c["batch"], c["heads"], d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c["batch"], c["length"], c["ragged"])):
        low = 0 if c["left"] < 0 else max(0, n - 1 - c["left"])
        keys = torch.cat([torch.arange(min(c["sinks"], low)), torch.arange(low, n)]).cuda()
        page, slot = s["table"][b].long()[keys // c["page"]], keys % c["page"]
        seen = torch.ones(share, keys.numel(), dtype=torch.bool, device="cuda")
        for h in range(c["kv_heads"]):
            out[b, h * share:(h + 1) * share] = _softmax_rows(
                s["q"][b, h * share:(h + 1) * share].double(), s["k"][0, :, h][page, slot].double(),
                s["v"][0, :, h][page, slot].double(), seen)
    return out.reshape(c["batch"], -1)
