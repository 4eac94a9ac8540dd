"""Steps and prefills of live streams behind a cache operation that failed: the old lengths are
still there, and nothing that the cache holds may be written over."""
import pytest
import torch

from gpu_util import rel_l2, to64, weights

pytestmark = pytest.mark.gpu

LAYERS, WIDTH, HEADS, HD = 2, 1280, 10, 128


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _start(api, dw, page=8):
    """Three streams of 20, 13 and 20 positions (2 is a fork of 0: they share a partly filled page);
    seven pages for the two that differ, five of them in use."""
    g = torch.Generator(device="cuda").manual_seed(page)
    cache = api.PagedCache.empty(LAYERS, 7, HEADS, page, HD, 3, 9)
    for pool in (cache.k, cache.v):
        pool.copy_(torch.randn(pool.shape, generator=g, device="cuda"))
    api.sal_cache_resize(cache, _ints([0, 1]), _ints([20, 13]))
    x = torch.randn(2, 20, WIDTH, generator=g, device="cuda")
    api.sal_stream_prefill(x.clone(), dw, LAYERS, cache, lengths=_ints([20, 13]), seqs=_ints([0, 1]))
    api.sal_cache_fork(cache, _ints([0]), _ints([2]))
    cache.check()
    return cache, g, x


def _fail(api, cache, how):
    if how == "pages":   # each of the three wants a page or a copy more, and then some: too many in all
        api.sal_cache_resize(cache, _ints([0, 1, 2]), _ints([21, 14, 60]))
    elif how == "list":  # a sequence twice
        api.sal_cache_resize(cache, _ints([0, 1, 0]), _ints([21, 14, 21]))
    else:                # a fork of one that does not exist
        api.sal_cache_fork(cache, _ints([0, 5]), _ints([1, 0]))


@pytest.mark.parametrize("how", ["pages", "list", "fork"])
@pytest.mark.parametrize("captured", [False, True])
def test_a_step_behind_a_failure_keeps_nothing(how, captured):
    api = _api()
    _, _, dw = weights(LAYERS)
    cache, g, x = _start(api, dw)
    before = [t.clone() for t in (cache.k, cache.v, cache.table, cache.lengths)]
    row = torch.randn(3, WIDTH, generator=g, device="cuda")
    emb, ws = torch.zeros(3, WIDTH, dtype=torch.bfloat16, device="cuda"), api.stream_workspace(3)
    scratch = api.PagedCache.empty(LAYERS, 7, HEADS, 8, HD, 3, 9)  # first calls outside a capture
    api.sal_cache_resize(scratch, _ints([0, 1, 2]), _ints([1, 1, 1]))
    api.sal_stream_step(row.clone(), dw, LAYERS, scratch, emb=emb, workspace=ws)
    _fail(api, cache, how)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.sal_stream_step(row, dw, LAYERS, cache, emb=emb, workspace=ws)
        graph.replay()
    else:
        api.sal_stream_step(row.clone(), dw, LAYERS, cache, emb=emb, workspace=ws)
    for a, b in zip((cache.k, cache.v, cache.table, cache.lengths), before):
        assert torch.equal(a, b)
    api.sal_stream_prefill(torch.randn_like(x), dw, LAYERS, cache, seqs=_ints([0, 1]))
    for a, b in zip((cache.k, cache.v, cache.table, cache.lengths), before):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError):
        cache.check()
    # cleared, and with room: the streams go on from what they had
    api.sal_cache_resize(cache, _ints([2, 0, 1]), _ints([0, 21, 14]))
    new = torch.randn(2, WIDTH, generator=g, device="cuda")
    got = api.sal_stream_step(new.clone(), dw, LAYERS, cache, seqs=_ints([0, 1]))
    cache.check()
    longer = torch.cat([x, torch.zeros(2, 1, WIDTH, device="cuda")], 1)
    longer[0, 20], longer[1, 13] = new[0], new[1]
    fresh = api.PagedCache.empty(LAYERS, 7, HEADS, 8, HD, 2, 9)
    api.sal_cache_resize(fresh, _ints([0, 1]), _ints([21, 14]))
    want = api.sal_stream_prefill(longer, dw, LAYERS, fresh, lengths=_ints([21, 14]))
    assert rel_l2(to64(got[0]), to64(want[0, 20])) < 1e-2 and rel_l2(to64(got[1]), to64(want[1, 13])) < 1e-2


def test_the_append_of_a_user_is_not_held_back():
    """It names its positions itself: those that are there are written, whatever failed before."""
    api = _api()
    _, _, dw = weights(LAYERS)
    cache, _, _ = _start(api, dw)
    _fail(api, cache, "pages")
    k = torch.randn(1, HEADS, 3, HD, device="cuda").bfloat16()
    api.sal_cache_append(cache, k, -k, _ints([11]), _ints([1]))  # 11 and 12 are there, 13 is not
    page = int(cache.table[1, 1])
    assert torch.equal(cache.k[0, page, :, 3:5], k[0, :, :2]) and torch.equal(cache.v[0, page, :, 3:5], -k[0, :, :2])
