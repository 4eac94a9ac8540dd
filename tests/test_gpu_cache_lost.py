"""Sequences cut back behind their window: positions in a page that has been let go stay lost. A
growth from the inside of such a page is refused (nothing changes), one from a page's edge is not."""
import random

import pytest
import torch

from stream_ref import CacheModel, attention_bound, paged_reference

pytestmark = pytest.mark.gpu

LOST = 4


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Model(CacheModel):
    """With the refusal, which comes before that of too few pages."""

    refused = 0

    def resize(self, seqs, new, left=-1, sinks=0):
        good = len(set(seqs)) == len(seqs) and all(0 <= s < self.sequences for s in seqs) and \
            all(0 <= n <= self.max_pages * self.page for n in new)
        for s, n in zip(seqs, new) if good else ():
            kept = min(max(0, self.lengths[s]), n)
            c = kept // self.page
            gone = left >= 0 and (c + 1) * self.page - 1 < kept - left and c * self.page >= sinks
            if n > kept and kept % self.page and (gone or not 0 <= self.table[s][c] < self.pages):
                self.status |= LOST
                self.refused += 1
                return
        super().resize(seqs, new, left, sinks)


def test_growth_behind_the_window_is_refused():
    """100 positions with ten visible, cut back to 40 (in a page that is gone): 41 is refused, in place
    and into other tables; from 32 or 48 on the sequence grows, and sees only what is its own."""
    api = _api()
    assert api.CACHE_LOST == LOST
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = api.PagedCache.empty(1, 12, 2, 16, 64, 2, 8)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    api.sal_cache_resize(cache, _ints([0, 1]), _ints([100, 50]))
    api.sal_cache_append(cache, rnd(2, 2, 100, 64), rnd(2, 2, 100, 64), _ints([0, 0]))
    api.sal_cache_resize(cache, _ints([1]), _ints([0]))       # sequence 1 leaves its pages
    api.sal_cache_resize(cache, _ints([0]), _ints([100]), 10)  # entries 0 to 4 are let go
    free = torch.ones(12, dtype=torch.bool, device="cuda")
    free[cache.table[cache.table >= 0].long()] = False
    cache.k[:, free], cache.v[:, free] = float("nan"), float("inf")
    api.sal_cache_resize(cache, _ints([0]), _ints([40]), 10)
    cache.check()
    before = [t.clone() for t in (cache.table, cache.lengths)]
    other = cache.with_tables(torch.full_like(cache.table, 99), torch.full_like(cache.lengths, 99))
    for out in (None, other):
        got = api.sal_cache_resize(cache, _ints([1, 0]), _ints([20, 41]), 10, out=out)
        assert int(cache.status.item()) == LOST
        assert torch.equal(got.table, before[0]) and torch.equal(got.lengths, before[1])
        with pytest.raises(RuntimeError, match="let go"):
            cache.check()
    q = rnd(2, 4, 64)
    for start in (32, 48):
        api.sal_cache_resize(cache, _ints([0]), _ints([start]), 10)
        for n in range(start + 1, start + 5):
            api.sal_cache_resize(cache, _ints([0]), _ints([n]), 10)
            api.sal_cache_append(cache, rnd(1, 2, 1, 64), rnd(1, 2, 1, 64), _ints([n - 1]), _ints([0]))
            o = api.sal_attention_paged(q, cache, 10).double().reshape(2, 4, 64)
            ref, spread = paged_reference(q, cache.k[0], cache.v[0], cache.table, cache.lengths, 10, 0)
            assert float(((o - ref).abs() - attention_bound(ref, spread)).max()) <= 0, n
        if start == 32:  # and once more from a page's edge further on
            api.sal_cache_resize(cache, _ints([0]), _ints([48]), 10)
            cache.check()
            api.sal_cache_append(cache, rnd(1, 2, 16, 64), rnd(1, 2, 16, 64), _ints([32]), _ints([0]))
    cache.check()


@pytest.mark.parametrize("seed", range(6))
def test_random_programs_behind_the_window(seed):
    """Windows of a few positions and cuts of many: tables, lengths and status after every call."""
    api, r = _api(), random.Random(100 + seed)
    page, n_seq, max_pages = r.choice([8, 16]), r.randint(1, 6), r.randint(4, 9)
    m = Model(r.randint(20, 60), page, n_seq, max_pages)
    c = api.PagedCache.empty(1, m.pages, 1, page, 64, n_seq, max_pages)
    for _ in range(60):
        some = r.sample(range(n_seq), r.randint(1, n_seq))
        new = [max(0, min(page * max_pages, m.lengths[s] + r.choice([1, 1, 5, 3 * page, -3, -2 * page, -4 * page])))
               for s in some]
        left, sinks = r.choice([(-1, 0), (r.randint(0, 2 * page), r.choice([0, 0, 3]))])
        api.sal_cache_resize(c, _ints(some), _ints(new), left, sinks)
        m.resize(some, new, left, sinks)
        if r.random() < 0.2:
            src = [r.randrange(n_seq) for _ in some]
            api.sal_cache_fork(c, _ints(src), _ints(some))
            m.fork(src, some)
        assert c.table.cpu().tolist() == m.table and c.lengths.cpu().tolist() == m.lengths
        assert int(c.status.item()) == m.status
        if r.random() < 0.2:
            c.status.zero_()
            m.status = 0
    assert m.refused > 0
