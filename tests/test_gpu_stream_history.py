"""Live streams step by step against the 64-bit attention over each stream's recorded history: a
key that is missing, stale or another stream's exceeds the bound. And scores of the windowed
attention that are infinite, as the paged attention's tests have them."""
import pytest
import torch

from stream_ref import attend, attention_bound, visible, window_reference

pytestmark = pytest.mark.gpu


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("H,kvh,d,page,left,sinks", [(10, 10, 128, 16, 40, 3), (8, 2, 64, 8, -1, 0),
                                                     (4, 4, 128, 32, 20, 0), (32, 2, 128, 64, 70, 17)])
def test_every_step_sees_its_own_history(H, kvh, d, page, left, sinks):
    """Forks, an end and a new start, a cut inside the window, pages let go, compaction, a captured
    step in the middle: every row of every step within the bound of one bf16 kernel."""
    api = _api()
    g = torch.Generator(device="cuda").manual_seed(page + d)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    S, layers, T, share = 5, 2, 70, H // kvh
    cache = api.PagedCache.empty(layers, 200, kvh, page, d, S, 40)
    cache.k.fill_(float("nan")), cache.v.fill_(float("inf"))  # what nobody has written
    lens = [70, 1, 33, 0, 64]
    k, v = rnd(layers, S, kvh, T, d), rnd(layers, S, kvh, T, d)
    api.sal_cache_resize(cache, _ints(list(range(S))), _ints(lens), left, sinks)
    for layer in range(layers):
        api.sal_cache_append(cache, k[layer], v[layer], _ints([0] * S), layer=layer)
    hist = [[[k[la, s, :, :n], v[la, s, :, :n]] for la in range(layers)] for s, n in enumerate(lens)]
    gone = [set() for _ in range(S)]  # positions whose pages the window let go

    def let_go(rows, kept):
        for s, n in zip(rows, kept):
            for c in range(n // page + 1):
                if left >= 0 and (c + 1) * page - 1 < n - left and c * page >= sinks:
                    gone[s] |= set(range(c * page, (c + 1) * page))

    def check(rows, layer, seqs, x, o):
        worst = 0.0
        for i, s in enumerate(rows):
            kk, vv = hist[s][layer]
            n = kk.shape[1]
            j = torch.arange(n)
            seen = visible(n - 1, j, n, left, 0, sinks) & ~torch.isin(j, torch.tensor(sorted(gone[s]), dtype=torch.int64))
            for h in range(kvh):
                ref, spread = attend(x[i, h * share:(h + 1) * share], kk[h], vv[h], seen.expand(share, n))
                off = (o[i, h * share:(h + 1) * share].double() - ref).abs() - attention_bound(ref, spread)
                worst = max(worst, float(off.max()))
        assert worst <= 0, (rows, layer, worst)

    for step in range(40):
        if step == 5:   # stream 2 goes on as 0 as well
            api.sal_cache_fork(cache, _ints([2]), _ints([0]))
            hist[0], gone[0] = [list(p) for p in hist[2]], set(gone[2])
        if step == 11:  # stream 4 ends, and starts again with the next position
            api.sal_cache_resize(cache, _ints([4]), _ints([0]))
            hist[4], gone[4] = [[a[:, :0] for a in p] for p in hist[4]], set()
        if step in (15, 28):  # stream 1 takes its last three positions back
            n = hist[1][0][0].shape[1] - 3
            api.sal_cache_resize(cache, _ints([1]), _ints([n]), left, sinks)
            let_go([1], [n])
            hist[1] = [[a[:, :n] for a in p] for p in hist[1]]
        if step in (17, 30):
            api.sal_cache_compact(cache)
        rows = [0, 1, 2, 4] if step % 3 else [3, 2, 0]
        old = [hist[s][0][0].shape[1] for s in rows]
        api.sal_cache_resize(cache, _ints(rows), _ints([n + 1 for n in old]), left, sinks)
        let_go(rows, old)
        for layer in range(layers):
            nk, nv, x = rnd(len(rows), kvh, 1, d), rnd(len(rows), kvh, 1, d), rnd(len(rows), H, d)
            for i, s in enumerate(rows):
                hist[s][layer] = [torch.cat([a, b[i]], 1) for a, b in zip(hist[s][layer], (nk, nv))]
            starts, seqs = _ints(old), _ints(rows)
            o = torch.zeros(len(rows), H * d, dtype=torch.bfloat16, device="cuda")
            ws = api.attention_paged_workspace(cache, len(rows), H)

            def run():
                api.sal_cache_append(cache, nk, nv, starts, seqs, layer)
                api.sal_attention_paged(x, cache, left, sinks, layer, seqs, o, ws)

            if step == 20:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    run()
                graph.replay()
            else:
                run()
            check(rows, layer, seqs, x, o.reshape(len(rows), H, d))
    cache.check()


def test_the_bound_notices_one_key():
    """Among 40 to 120 keys one that is left out, or another's value, is over the bound somewhere."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for n in (40, 120):
        for trial in range(20):
            q, k, v = (torch.randn(m, 128, generator=g, device="cuda").bfloat16() for m in (10, n, n))
            seen = torch.ones(10, n, dtype=torch.bool)
            ref, spread = attend(q, k, v, seen)
            seen[:, trial] = False
            less, _ = attend(q, k, v, seen)
            v[trial] = torch.randn(128, generator=g, device="cuda").bfloat16()
            other, _ = attend(q, k, v, torch.ones(10, n, dtype=torch.bool))
            for wrong in (less, other):
                assert bool(((wrong - ref).abs() > attention_bound(ref, spread)).any())


@pytest.mark.parametrize("T,H,kvh,d,left,right,sinks", [(300, 2, 2, 128, 200, 0, 0), (700, 4, 2, 64, -1, -1, 0),
                                                        (900, 3, 3, 64, 130, 5, 3), (2100, 8, 2, 128, 150, 0, 4)])
def test_windowed_scores_that_are_infinite(T, H, kvh, d, left, right, sinks):
    """Keys whose score is -infinity have a weight of zero, whole tiles of them too; a row that sees no
    other, and one that sees a score of +infinity, is no number."""
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(2, h, T, d, generator=g, device="cuda").bfloat16() for h in (H, kvh, kvh))
    q[..., 5] = 1.0
    low = torch.zeros(T, dtype=torch.bool)
    low[:T // 2:2] = low[T // 2:] = low[3] = True
    high = T // 4
    k[0][:, low.cuda(), 5] = float("-inf")
    k[1, :, high, 5] = float("inf")
    o = _api().sal_attention_window(q, k, v, left, right, sinks).double().reshape(2, T, H, d)
    p, j = torch.arange(T)[:, None], torch.arange(T)[None, :]
    seen = visible(p, j, T, left, right, sinks).expand(T, T)
    some = (seen & ~low).any(1)
    assert bool(torch.isnan(o[0][~some.cuda()]).all()) and bool(torch.isnan(o[1][seen[:, high].cuda()]).all())
    share = H // kvh
    for h in range(H):
        ref, spread = attend(q[0, h], k[0, h // share], v[0, h // share], seen & ~low)
        off = (o[0, :, h] - ref).abs() - attention_bound(ref, spread)
        assert bool((off[some.cuda()] <= 0).all())
    ref, spread = window_reference(q[1:], k[1:], v[1:], left, right, sinks, [T])
    off = (o[1] - ref[0]).abs() - attention_bound(ref[0], spread[0])
    assert bool((off[~seen[:, high].cuda()] <= 0).all())
