"""The page operations of the cache against the step-by-step model (stream_ref.CacheModel):
every table, length, status bit and page must be equal. Page contents are labels, so a copy
that misses a layer, a head or a vector shows."""
import random

import pytest
import torch

from stream_ref import CacheModel

pytestmark = pytest.mark.gpu


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Pair:
    """A cache on the GPU beside the model. Position labels are small integers; slot s of head
    h of layer l holds, in element e, bf16(label) + a pattern of (l, h, e) that bf16 keeps."""

    def __init__(self, layers=2, pages=40, kv_heads=3, page=8, head_dim=64, sequences=6, max_pages=9, seed=0):
        api = _api()
        self.m = CacheModel(pages, page, sequences, max_pages)
        self.c = api.PagedCache.empty(layers, pages, kv_heads, page, head_dim, sequences, max_pages)
        self.layers, self.kvh, self.page, self.hd = layers, kv_heads, page, head_dim
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.c.k.copy_(torch.randn(self.c.k.shape, generator=g, device="cuda"))
        self.c.v.copy_(torch.randn(self.c.v.shape, generator=g, device="cuda"))
        self.rows = {}  # label -> (k, v) [layers, kv_heads, head_dim]
        for p in range(pages):
            for s in range(page):
                x = ("start", p, s)
                self.rows[x] = (self.c.k[:, p, :, s].clone(), self.c.v[:, p, :, s].clone())
                self.m.data[p][s] = x
        self.g, self.next = g, 0

    def new_tokens(self, batch, T):
        k = torch.randn(self.layers, batch, self.kvh, T, self.hd, generator=self.g, device="cuda").bfloat16()
        v = torch.randn(self.layers, batch, self.kvh, T, self.hd, generator=self.g, device="cuda").bfloat16()
        labels = []
        for b in range(batch):
            labels.append([])
            for t in range(T):
                self.rows[self.next] = (k[:, b, :, t], v[:, b, :, t])
                labels[b].append(self.next)
                self.next += 1
        return k, v, labels

    def append(self, starts, T, seqs=None):
        api = _api()
        k, v, labels = self.new_tokens(len(starts), T)
        for layer in range(self.layers):
            api.sal_cache_append(self.c, k[layer], v[layer], _ints(starts), None if seqs is None else _ints(seqs), layer)
        self.m.append(labels, starts, seqs)

    def agree(self, cache=None):
        c = self.c if cache is None else cache
        assert c.table.cpu().tolist() == self.m.table
        assert c.lengths.cpu().tolist() == self.m.lengths
        assert int(c.status.item()) == self.m.status
        want_k, want_v = torch.empty_like(c.k), torch.empty_like(c.v)
        want_k[:] = torch.stack([torch.stack([self.rows[x][0] for x in p], 2) for p in self.m.data], 1)
        want_v[:] = torch.stack([torch.stack([self.rows[x][1] for x in p], 2) for p in self.m.data], 1)
        assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)


def test_grow_append_cut_free():
    api, p = _api(), Pair()
    for seqs, new in (([0, 3], [5, 17]), ([3, 0], [8, 24]), ([1], [1]), ([0], [0]), ([2, 0, 5], [72, 9, 3])):
        starts = [p.m.lengths[s] for s in seqs]
        api.sal_cache_resize(p.c, _ints(seqs), _ints(new))
        p.m.resize(seqs, new)
        p.append([min(a, n) for a, n in zip(starts, new)], 20, seqs)
        p.agree()


def test_append_skips_what_has_no_place():
    """Tokens before 0 and past the length, sequences out of range and let-go pages."""
    api, p = _api(), Pair()
    api.sal_cache_resize(p.c, _ints([0, 1, 2]), _ints([20, 9, 30]))
    p.m.resize([0, 1, 2], [20, 9, 30])
    p.c.table[2, 1] = p.m.table[2][1] = -1
    p.c.table[2, 2] = p.m.table[2][2] = 1000
    p.append([-3, 5, 0, 0, 0, 2 ** 31 - 2], 30, [0, 1, 2, -1, 77, 3])
    p.agree()
    p.append([2, 8, -1, 0, 0, 0], 7)  # row b is sequence b
    p.agree()


def test_copy_pages_and_bad_pairs():
    api, p = _api(), Pair(layers=3, page=16, head_dim=128, kv_heads=5)
    src, dst = [0, 1, 0, 39, 40, 5, -1], [7, 8, 9, 10, 11, 99, 12]
    api.sal_cache_copy_pages(p.c, _ints(src), _ints(dst))
    p.m.copy(src, dst)
    p.agree()
    assert p.m.status == CacheModel.BAD_LIST
    with pytest.raises(RuntimeError):
        p.c.check()
    p.c.check()  # cleared


def test_fork_permutes_and_multiplies_in_place():
    api, p = _api(), Pair()
    new = [5, 17, 24, 0, 33, 8]
    api.sal_cache_resize(p.c, _ints(list(range(6))), _ints(new))
    p.m.resize(list(range(6)), new)
    for src, dst in (([1, 0], [0, 1]), ([2, 2, 4, 3], [0, 2, 3, 5]), ([5, 4, 3, 2, 1, 0], [0, 1, 2, 3, 4, 5]), ([], [])):
        api.sal_cache_fork(p.c, _ints(src), _ints(dst))
        p.m.fork(src, dst)
        p.agree()


@pytest.mark.parametrize("src,dst", [([0, 1], [2, 2]), ([6], [0]), ([0], [-1]), ([-1], [0]), ([0], [6])])
def test_fork_refuses_on_the_device(src, dst):
    api, p = _api(), Pair()
    api.sal_cache_resize(p.c, _ints([0, 1]), _ints([9, 20]))
    p.m.resize([0, 1], [9, 20])
    api.sal_cache_fork(p.c, _ints(src), _ints(dst))
    p.m.fork(src, dst)
    assert p.m.status == CacheModel.BAD_LIST
    p.agree()
    other = p.c.with_tables(torch.full_like(p.c.table, 99), torch.full_like(p.c.lengths, 99))
    api.sal_cache_fork(p.c, _ints(src), _ints(dst), out=other)
    p.agree(other)


@pytest.mark.parametrize("seqs,new", [([0, 0], [3, 4]), ([6], [1]), ([-1], [1]), ([2], [73]), ([2], [-1]),
                                      ([2, 3, 4, 5], [72, 72, 72, 72])])
def test_resize_refuses_on_the_device(seqs, new):
    """A bad list, and more pages than are free: nothing changes, in place or into other tables."""
    api, p = _api(), Pair(pages=30)
    api.sal_cache_resize(p.c, _ints([0, 1]), _ints([9, 20]))
    p.m.resize([0, 1], [9, 20])
    api.sal_cache_resize(p.c, _ints(seqs), _ints(new))
    p.m.resize(seqs, new)
    assert p.m.status != 0
    p.agree()
    other = p.c.with_tables(torch.full_like(p.c.table, 99), torch.full_like(p.c.lengths, 99))
    api.sal_cache_resize(p.c, _ints(seqs), _ints(new), out=other)
    p.agree(other)
    # and a row that did not grow writes nothing
    p.append([9, 20], 3, [0, 1])
    p.agree(other)


def test_exactly_all_pages():
    api, p = _api(), Pair(pages=33, sequences=4, max_pages=9)
    for new in ([72, 72, 72, 48], [72, 72, 72, 49], [0, 72, 72, 72]):
        api.sal_cache_resize(p.c, _ints([0, 1, 2, 3]), _ints(new))
        p.m.resize([0, 1, 2, 3], new)
        p.agree()
    assert p.m.status == CacheModel.NO_PAGES


def test_growth_of_shared_pages_copies_them():
    api, p = _api(), Pair(layers=4, kv_heads=2, page=16, head_dim=128, pages=64)
    api.sal_cache_resize(p.c, _ints([0]), _ints([37]))
    p.m.resize([0], [37])
    p.append([0], 37, [0])
    for src, dst, seqs, new in (([0, 0, 0], [1, 2, 3], [1, 2], [38, 50]), ([1, 3], [4, 5], [0, 3, 5, 4], [40, 38, 49, 39]),
                                ([4, 4], [0, 1], [0, 1, 4], [20, 17, 16]), ([], [], [0, 1, 4], [21, 18, 17])):
        api.sal_cache_fork(p.c, _ints(src), _ints(dst))
        p.m.fork(src, dst)
        starts = [p.m.lengths[s] for s in seqs]
        api.sal_cache_resize(p.c, _ints(seqs), _ints(new))
        p.m.resize(seqs, new)
        p.append([min(a, n) for a, n in zip(starts, new)], 4, seqs)
        p.agree()


@pytest.mark.parametrize("left,sinks", [(0, 0), (10, 0), (10, 3), (7, 20), (100, 0)])
def test_window_lets_pages_go(left, sinks):
    api, p = _api(), Pair(sequences=3, max_pages=12, pages=30)
    new = [0, 0, 0]
    for step in range(14):
        starts = list(new)
        new = [min(96, n + a) for n, a in zip(new, (7, 1, 16))]
        api.sal_cache_resize(p.c, _ints([2, 0, 1]), _ints([new[2], new[0], new[1]]), left=left, sinks=sinks)
        p.m.resize([2, 0, 1], [new[2], new[0], new[1]], left, sinks)
        p.append(starts, 16)
        p.agree()
        new = list(p.m.lengths)


def test_compact():
    api, p = _api(), Pair(layers=3, page=16, pages=70, sequences=8, max_pages=9)
    api.sal_cache_compact(p.c)
    p.agree()  # an empty cache
    new = [100, 3, 40, 0, 77, 144, 16, 20]
    api.sal_cache_resize(p.c, _ints(list(range(8))), _ints(new))
    p.m.resize(list(range(8)), new)
    p.append([0] * 8, 144)
    api.sal_cache_resize(p.c, _ints([0, 2, 5]), _ints([0, 17, 120]))
    p.m.resize([0, 2, 5], [0, 17, 120])
    api.sal_cache_fork(p.c, _ints([7]), _ints([3]))
    p.m.fork([7], [3])
    p.agree()
    old = p.c.with_tables(p.c.table.clone(), p.c.lengths.clone())
    other = p.c.with_tables(torch.full_like(p.c.table, 99), torch.full_like(p.c.lengths, 99))
    api.sal_cache_compact(p.c, out=other)
    assert torch.equal(p.c.table, old.table)
    p.m.compact()
    p.agree(other)
    api.sal_cache_compact(other)  # nothing left to move
    p.m.compact()
    p.agree(other)


@pytest.mark.parametrize("seed", range(8))
def test_random_programs(seed):
    """Thirty operations in a row, in place or into other tables, against the model."""
    api, r = _api(), random.Random(seed)
    page = r.choice([8, 16, 32])
    p = Pair(layers=r.choice([1, 3]), pages=r.randint(20, 120), kv_heads=r.randint(1, 4), page=page,
             head_dim=r.choice([64, 128]), sequences=r.randint(1, 40), max_pages=r.randint(1, 12), seed=seed)
    n_seq, cap = p.m.sequences, p.m.max_pages * page
    spare = p.c.with_tables(torch.zeros_like(p.c.table), torch.zeros_like(p.c.lengths))
    for _ in range(30):
        op = r.choice(["resize", "resize", "fork", "compact", "append", "copy"])
        out = r.choice([None, spare])
        some = r.sample(range(n_seq), r.randint(0, n_seq))
        if op == "resize":
            new = [max(0, min(cap, p.m.lengths[s] + r.choice([1, 1, 5, page, -3, -page, -cap]))) for s in some]
            left, sinks = r.choice([(-1, 0), (-1, 0), (r.randint(0, cap), r.randint(0, 20))])
            got = api.sal_cache_resize(p.c, _ints(some), _ints(new), left, sinks, out)
            p.m.resize(some, new, left, sinks)
        elif op == "fork":
            src = [r.randrange(n_seq) for _ in some]
            got = api.sal_cache_fork(p.c, _ints(src), _ints(some), out)
            p.m.fork(src, some)
        elif op == "compact":
            got = api.sal_cache_compact(p.c, out)
            p.m.compact()
        elif op == "append":
            # positions that no other sequence on the list shares, so the result has one meaning
            shared = p.m.counts()
            ok = [s for s in some if p.m.lengths[s] and
                  shared[max(0, p.m.table[s][(p.m.lengths[s] - 1) // page])] == 1]
            if ok:
                p.append([p.m.lengths[s] - 1 for s in ok], 2, ok)
            got = p.c
        else:
            free = [x for x, c in enumerate(p.m.counts()) if c == 0]
            used = [x for x, c in enumerate(p.m.counts()) if c]
            k = min(len(free), len(used), 3)
            api.sal_cache_copy_pages(p.c, _ints(used[:k]), _ints(free[:k]))
            p.m.copy(used[:k], free[:k])
            got = p.c
        p.agree(got)
        if got is not p.c:
            p.c, spare = got, p.c


def test_the_largest_tables():
    """524,288 pages and 32,768 sequences (one small head): the bitmaps at their full size, a list
    of every sequence, in-place fork by a permutation."""
    api = _api()
    pages, seqs = 524288, 32768
    c = api.PagedCache.empty(1, pages, 1, 8, 64, seqs, 20)
    every = torch.arange(seqs, dtype=torch.int32, device="cuda")
    api.sal_cache_resize(c, every, torch.full_like(every, 121))  # 16 pages each: all of them
    c.check()
    assert torch.equal(c.table[:, :16].reshape(-1), torch.arange(pages, dtype=torch.int32, device="cuda"))
    assert bool((c.table[:, 16:] == -1).all())
    api.sal_cache_resize(c, every[:1], torch.full_like(every[:1], 129))
    assert int(c.status.item()) == api.CACHE_NO_PAGES
    c.status.zero_()
    api.sal_cache_fork(c, every.flip(0).contiguous(), every)
    assert torch.equal(c.table[:, :16].flip(0).reshape(-1), torch.arange(pages, dtype=torch.int32, device="cuda"))
    api.sal_cache_resize(c, every[::2].contiguous(), torch.zeros_like(every[::2]))
    api.sal_cache_compact(c)
    c.check()
    used = c.table[1::2, :16].reshape(-1)
    assert torch.equal(used.sort().values, torch.arange(pages // 2, dtype=torch.int32, device="cuda"))
    # sequences that lay in the lower half have not moved
    stay = torch.arange(pages, dtype=torch.int32, device="cuda").reshape(seqs, 16).flip(0)[1::2]
    low = stay[:, 0] < pages // 2
    assert torch.equal(c.table[1::2, :16][low], stay[low])


def test_a_list_that_asks_for_more_than_32_bits_of_pages():
    """64 sequences that each ask for 2^25 pages: 2^31 in all, of the 40 there are."""
    api = _api()
    c = api.PagedCache.empty(1, 40, 1, 8, 64, 65, 1 << 25)
    api.sal_cache_resize(c, _ints([64]), _ints([20]))
    c.check()
    for n in (63, 64):
        api.sal_cache_resize(c, _ints(range(n)), _ints([1 << 28] * n))
        assert int(c.status.item()) == api.CACHE_NO_PAGES
        c.status.zero_()
        assert c.lengths.tolist() == [0] * 64 + [20] and c.table[64, :4].tolist() == [0, 1, 2, -1]
        assert int(c.table[0].max()) == -1
    del c
    torch.cuda.empty_cache()


def test_pages_past_32_bits():
    """A pool of 2.7 G elements: pages in its last gigabyte are written, copied and moved."""
    api = _api()
    pages, H, ps, hd = 132000, 10, 16, 128
    c = api.PagedCache(torch.zeros(1, pages, H, ps, hd, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(1, pages, H, ps, hd, dtype=torch.bfloat16, device="cuda"),
                       _ints([[pages - 1, pages - 3]]), _ints([32]))
    k = torch.randn(1, H, 32, hd, device="cuda").bfloat16()
    v = torch.randn(1, H, 32, hd, device="cuda").bfloat16()
    api.sal_cache_append(c, k, v, _ints([0]))
    for pool, x in ((c.k, k), (c.v, v)):
        assert torch.equal(pool[0, pages - 1], x[0, :, :16]) and torch.equal(pool[0, pages - 3], x[0, :, 16:])
    api.sal_cache_copy_pages(c, _ints([pages - 1]), _ints([pages - 2]))
    assert torch.equal(c.k[0, pages - 2], k[0, :, :16]) and torch.equal(c.v[0, pages - 2], v[0, :, :16])
    api.sal_cache_compact(c)
    # the used pages in ascending order: pages - 3 (entry 1) moves to 0, pages - 1 to 1
    assert c.table.cpu().tolist() == [[1, 0]]
    assert torch.equal(c.k[0, 1], k[0, :, :16]) and torch.equal(c.v[0, 0], v[0, :, 16:])


def test_captured_and_replayed():
    """resize, append and compact in one graph: the lists are read at replay."""
    api, p = _api(), Pair()
    seqs, new, starts = _ints([0, 1]), _ints([6, 3]), _ints([0, 0])
    k, v, labels = p.new_tokens(2, 12)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # first calls outside a capture
        spare = p.c.with_tables(p.c.table.clone(), p.c.lengths.clone())
        api.sal_cache_resize(spare, seqs, new)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.sal_cache_resize(p.c, seqs, new)
        for layer in range(p.layers):
            api.sal_cache_append(p.c, k[layer], v[layer], starts, seqs, layer)
        api.sal_cache_compact(p.c)
    for s, n, st in (([0, 1], [6, 3], [0, 0]), ([5, 0], [11, 9], [0, 6]), ([1, 0], [0, 18], [0, 9])):
        for t, x in ((seqs, s), (new, n), (starts, st)):
            t.copy_(_ints(x))
        graph.replay()
        p.m.resize(s, n)
        p.m.append(labels, st, s)
        p.m.compact()
        p.agree()


def test_python_refusals():
    api, p = _api(), Pair()
    with pytest.raises(ValueError):
        api.sal_cache_fork(p.c, _ints([0, 1]), _ints([2]))
    with pytest.raises(ValueError):
        api.sal_cache_resize(p.c, torch.zeros(1, dtype=torch.int64, device="cuda"), _ints([2]))
    with pytest.raises(ValueError):
        api.sal_cache_resize(p.c, _ints([0]), _ints([2]), out=Pair().c)
    with pytest.raises(ValueError):
        p.c.with_tables(p.c.table[:2].contiguous(), p.c.lengths)
    k = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        api.sal_cache_append(p.c, k[:, :2].contiguous(), k, _ints([0]))
    with pytest.raises(api.SalError):
        api.sal_cache_append(p.c, k, k, _ints([0]), layer=2)
    with pytest.raises(api.SalError):
        api.sal_cache_resize(p.c, _ints([0] * 7), _ints([0] * 7))
