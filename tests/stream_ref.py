"""Plain 64-bit forms of the windowed and the paged attention and a step-by-step model of
the page tables, for the tests of the live-stream calls (no test functions here)."""
from __future__ import annotations

import torch

BF16_HALF_STEP = 2.0 ** -8  # a bf16 rounding is off by at most this, relative to the value


def visible(p, j, n: int, left: int, right: int, sinks: int):
    """Whether key j is visible to position p of n (broadcasting integer tensors)."""
    ok = (j >= 0) & (j < n)
    if right >= 0:
        ok = ok & (j <= p + right)
    if left >= 0:
        ok = ok & ((j >= p - left) | (j < sinks))
    return ok


def attend(q, k, v, seen):
    """(softmax(q k^T / sqrt(d)) v, the same weights over |v|) in 64 bits over the keys that
    `seen` allows; rows that see nothing are zero. q [..., r, d], k and v [..., c, d]."""
    seen = seen.to(q.device)
    k = torch.where(torch.isfinite(k), k, 0.0).double()
    v = torch.where(torch.isfinite(v), v, 0.0).double()
    s = (q.double() @ k.transpose(-1, -2)) * q.shape[-1] ** -0.5
    s = s.masked_fill(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(torch.isinf(top), 0.0, top)).masked_fill(~seen, 0.0)
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return w @ v, w @ v.abs()


def attention_bound(ref, spread, q_scale: float = 1.0):
    """How far a kernel's bf16 output may be from `ref`, the 64-bit result, where `spread` =
    sum_j a_j |v_j|, for keys of unit variance and queries of standard deviation q_scale.

    Each weight is rounded to bf16 once before it meets its v (half a step, 2^-8 of it). Its
    fp32 score, in log2 units, is a sum of d <= 128 products times log2(e) / sqrt(d): off by
    at most d 2^-24 log2(e) / sqrt(d) sum |q_i k_i|, where sum |q_i k_i| is below d q_scale
    (0.64 d q_scale on average), so by at most 128^1.5 2^-24 1.45 q_scale < 2^-12 q_scale,
    and the weight by ln 2 of that; ex2.approx adds 2^-22. A sum of n fp32 terms adds n 2^-24,
    below 2^-14 at n = 1,024. Doubled for the normaliser (which sums the unrounded weights):
    2 (0.7 2^-12 + 2^-14) q_scale < 2^-10 q_scale. The output is rounded once more (half a
    step of it)."""
    rel = BF16_HALF_STEP + 2.0 ** -10 * q_scale
    return rel * spread + BF16_HALF_STEP * (ref.abs() + rel * spread) + 1e-30


def window_reference(q, k, v, left, right, sinks, lengths):
    """[batch, T, heads, d] results and spreads; rows past a length are NaN."""
    B, H, T, d = q.shape
    share = H // k.shape[1]
    out = torch.full((B, T, H, d), float("nan"), dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(out)
    for b in range(B):
        n = max(0, min(T, int(lengths[b])))
        if n == 0:
            continue
        p = torch.arange(n, device=q.device)[:, None]
        seen = visible(p, torch.arange(n, device=q.device)[None, :], n, left, right, sinks)
        for h in range(H):
            o, s = attend(q[b, h, :n], k[b, h // share, :n], v[b, h // share, :n], seen)
            out[b, :n, h], spread[b, :n, h] = o, s
    return out, spread


def paged_reference(q, k, v, table, lengths, left, sinks, seqs=None):
    """q [batch, heads, d], one layer's k and v [pages, kv_heads, page, d] -> [batch, heads, d] x 2."""
    B, H, d = q.shape
    pages, kvh, page, _ = k.shape
    out = torch.zeros(B, H, d, dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(out)
    table, lengths = table.cpu().tolist(), lengths.cpu().tolist()
    for b in range(B):
        s = b if seqs is None else int(seqs[b])
        if not 0 <= s < len(table):
            continue
        n = max(0, min(lengths[s], len(table[s]) * page))
        keys = [j for j in range(n) if 0 <= table[s][j // page] < pages and
                (left < 0 or j >= n - 1 - left or j < sinks)]
        if not keys:
            continue
        at = torch.tensor([table[s][j // page] for j in keys], device=q.device)
        slot = torch.tensor([j % page for j in keys], device=q.device)
        seen = torch.ones(H // kvh, len(keys), dtype=torch.bool)
        for h in range(kvh):
            rows = slice(h * (H // kvh), (h + 1) * (H // kvh))
            out[b, rows], spread[b, rows] = attend(q[b, rows], k[at, h, slot], v[at, h, slot], seen)
    return out, spread


class CacheModel:
    """The page tables, one step at a time: plain lists, the pages' contents as one label per
    (page, slot) that moves with them."""

    NO_PAGES, BAD_LIST = 1, 2

    def __init__(self, pages, page, sequences, max_pages):
        self.pages, self.page, self.sequences, self.max_pages = pages, page, sequences, max_pages
        self.table = [[-1] * max_pages for _ in range(sequences)]
        self.lengths = [0] * sequences
        self.data = [[None] * page for _ in range(pages)]
        self.status = 0

    def used_entries(self, s):
        return -(-max(0, min(self.lengths[s], self.max_pages * self.page)) // self.page)

    def counts(self):
        got = [0] * self.pages
        for s in range(self.sequences):
            for c in range(self.used_entries(s)):
                if 0 <= self.table[s][c] < self.pages:
                    got[self.table[s][c]] += 1
        return got

    def append(self, labels, starts, seqs=None):
        """labels[b][t] goes to position starts[b] + t of sequence seqs[b]."""
        for b, row in enumerate(labels):
            s = b if seqs is None else seqs[b]
            if not 0 <= s < self.sequences:
                continue
            for t, x in enumerate(row):
                p = starts[b] + t
                if 0 <= p < self.lengths[s] and 0 <= self.table[s][p // self.page] < self.pages:
                    self.data[self.table[s][p // self.page]][p % self.page] = x

    def copy(self, src, dst):
        for a, b in zip(src, dst):
            if 0 <= a < self.pages and 0 <= b < self.pages:
                self.data[b] = list(self.data[a])
            else:
                self.status |= self.BAD_LIST

    def fork(self, src, dst):
        everyone = range(self.sequences)
        if any(s not in everyone for s in src + dst) or len(set(dst)) != len(dst):
            self.status |= self.BAD_LIST
            return
        rows, lens = [list(self.table[s]) for s in src], [self.lengths[s] for s in src]
        for d, row, n in zip(dst, rows, lens):
            self.table[d], self.lengths[d] = row, n

    def resize(self, seqs, new, left=-1, sinks=0):
        capacity = self.max_pages * self.page
        if any(not 0 <= s < self.sequences for s in seqs) or len(set(seqs)) != len(seqs) or \
                any(not 0 <= n <= capacity for n in new):
            self.status |= self.BAD_LIST
            return
        before = [list(r) for r in self.table], list(self.lengths)
        kept = {}
        for s, n in zip(seqs, new):
            kept[s] = min(max(0, self.lengths[s]), n)
            self.lengths[s] = kept[s]
            for c in range(self.max_pages):
                first, last = c * self.page, c * self.page + self.page - 1
                gone = left >= 0 and last < kept[s] - left and first >= sinks
                if c >= self.used_entries(s) or gone or not 0 <= self.table[s][c] < self.pages:
                    self.table[s][c] = -1
        count = self.counts()
        free = [p for p in range(self.pages) if count[p] == 0]
        copies = []
        try:
            for s, n in zip(seqs, new):
                c = kept[s] // self.page
                if n > kept[s] and kept[s] % self.page:
                    old = self.table[s][c]
                    if old < 0 or count[old] > 1:
                        self.table[s][c] = free.pop(0)
                        if old >= 0:
                            copies.append((old, self.table[s][c]))
                for c in range(-(-kept[s] // self.page), -(-n // self.page)):
                    self.table[s][c] = free.pop(0)
                self.lengths[s] = n
        except IndexError:
            self.table, self.lengths = before
            self.status |= self.NO_PAGES
            return
        for a, b in copies:
            self.data[b] = list(self.data[a])

    def compact(self):
        count = self.counts()
        m = sum(1 for c in count if c)
        movers = [p for p in range(m, self.pages) if count[p]]
        holes = [p for p in range(m) if not count[p]]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.data[b] = list(self.data[a])
        for s in range(self.sequences):
            self.table[s] = [to.get(p, p) if c < self.used_entries(s) and 0 <= p < self.pages else -1
                             for c, p in enumerate(self.table[s])]
