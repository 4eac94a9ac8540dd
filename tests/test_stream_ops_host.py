"""Argument checks of the live-stream calls (windowed attention, paged cache, attention over
it): everything here returns before any CUDA call. And the tests' model of the page tables
against what sal.h states, by hand-worked cases."""
import ctypes

import pytest

from stream_ref import CacheModel

OK, EINVAL, ESHAPE, EWORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def api():
    from speech_audio_encoder_b200 import api as a
    from speech_audio_encoder_b200 import build
    build.build(quiet=True)
    return a


def _window(api, **kw):
    w = api.sal_window(kw.get("left", -1), kw.get("right", -1), kw.get("sinks", 0))
    return ctypes.byref(w)


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), EINVAL), (dict(T=-1), EINVAL), (dict(heads=-1), EINVAL), (dict(kv_heads=-1), EINVAL),
    (dict(T=0), OK), (dict(batch=0), OK), (dict(heads=0), OK),
    (dict(kv_heads=0), EINVAL), (dict(kv_heads=3), EINVAL), (dict(head_dim=96), ESHAPE), (dict(T=90001), ESHAPE),
    (dict(batch=6554), ESHAPE), (dict(q=0), EINVAL), (dict(k=0), EINVAL), (dict(v=0), EINVAL), (dict(o=0), EINVAL),
    (dict(q=4104), EINVAL), (dict(o=4097), EINVAL), (dict(lengths=4097), EINVAL), (dict(sinks=-1), EINVAL),
])
def test_window_attention_refusals(api, change, want):
    a = dict(q=4096, k=4096, v=4096, o=4096, lengths=0, batch=1, T=10, heads=10, kv_heads=10, head_dim=128, sinks=0)
    a.update(change)
    assert api.lib().sal_attention_window(a["q"], a["k"], a["v"], a["batch"], a["T"], a["heads"], a["kv_heads"],
                                          a["head_dim"], _window(api, sinks=a["sinks"]), a["lengths"], a["o"],
                                          0) == want


def test_window_withhold_refusals(api):
    f = api.lib().sal_attention_window_withhold
    assert f(4096, 4096, 4096, 1, 512, 4, 128, None, -1, 4096, 0) == EINVAL
    assert f(4096, 4096, 4096, 1, 512, 4, 96, None, 1, 4096, 0) == ESHAPE
    assert f(0, 4096, 4096, 1, 512, 4, 128, None, 1, 4096, 0) == EINVAL
    assert f(4096, 4096, 4096, 1, 0, 4, 128, None, 1, 4096, 0) == OK


def _cache(api, **change):
    c = dict(k=4096, v=4096, layers=2, pages=64, kv_heads=2, page_size=16, head_dim=128, sequences=4, max_pages=8,
             table=4096, lengths=4096, status=4096, workspace=4096, workspace_bytes=1 << 20)
    c.update(change)
    return api.sal_cache(*[c[n] for n, _ in api.sal_cache._fields_])


BAD_CACHES = [(dict(k=0), EINVAL), (dict(v=8), EINVAL), (dict(table=0), EINVAL), (dict(table=2), EINVAL),
              (dict(lengths=0), EINVAL), (dict(status=0), EINVAL), (dict(layers=-1), EINVAL), (dict(pages=-1), EINVAL),
              (dict(layers=0), ESHAPE), (dict(layers=32768), ESHAPE), (dict(pages=0), ESHAPE),
              (dict(pages=524289), ESHAPE), (dict(kv_heads=0), ESHAPE), (dict(page_size=4), ESHAPE),
              (dict(page_size=24), ESHAPE), (dict(page_size=512), ESHAPE), (dict(head_dim=32), ESHAPE),
              (dict(sequences=0), ESHAPE), (dict(sequences=32769), ESHAPE), (dict(max_pages=0), ESHAPE),
              (dict(max_pages=(1 << 24) + 1), ESHAPE)]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_every_cache_call_refuses_a_bad_record(api, change, want):
    lib, c = api.lib(), _cache(api, **change)
    r = ctypes.byref(c)
    assert lib.sal_cache_append(r, 0, 4096, 4096, 1, 1, 4096, 0, 0) == want
    assert lib.sal_cache_copy_pages(r, 4096, 4096, 1, 0) == want
    assert lib.sal_cache_fork(r, 4096, 4096, 1, 4096, 4096, 0) == want
    assert lib.sal_cache_resize(r, 4096, 4096, 1, None, 4096, 4096, 0) == want
    assert lib.sal_cache_compact(r, 4096, 4096, 0) == want
    assert lib.sal_attention_paged(4096, 256, 128, 1, 2, r, 0, 0, None, 4096, 4096, 1 << 30, 0) == want


def test_null_cache(api):
    lib = api.lib()
    assert lib.sal_cache_append(None, 0, 4096, 4096, 1, 1, 4096, 0, 0) == EINVAL
    assert lib.sal_cache_compact(None, 4096, 4096, 0) == EINVAL
    assert lib.sal_attention_paged(4096, 256, 128, 1, 2, None, 0, 0, None, 4096, 4096, 1 << 30, 0) == EINVAL
    assert lib.sal_attention_paged_workspace_bytes(None, 1, 2) == 0


def test_cache_call_refusals(api):
    lib, c = api.lib(), _cache(api)
    r = ctypes.byref(c)
    append = lambda layer=0, k=4096, v=4096, b=1, T=1, st=4096, sq=0: lib.sal_cache_append(r, layer, k, v, b, T, st, sq, 0)  # noqa: E731,E501
    assert append(layer=2) == EINVAL and append(layer=-1) == EINVAL and append(b=-1) == EINVAL and append(T=-1) == EINVAL
    assert append(b=0) == OK and append(T=0) == OK
    assert append(k=0) == EINVAL and append(v=4104) == EINVAL and append(st=4097) == EINVAL and append(sq=4098) == EINVAL
    assert append(b=5) == EINVAL            # five rows without a list, four sequences
    assert append(b=65536, sq=4096) == ESHAPE and append(T=(1 << 28) + 1) == ESHAPE
    assert append(T=(1 << 26) + 1) == ESHAPE  # 2 heads x T x 16 vectors past 2^31
    assert lib.sal_cache_copy_pages(r, 4096, 4096, 0, 0) == OK
    assert lib.sal_cache_copy_pages(r, 4096, 4096, -1, 0) == EINVAL
    assert lib.sal_cache_copy_pages(r, 4096, 4096, 65, 0) == EINVAL  # more pairs than pages
    assert lib.sal_cache_copy_pages(r, 0, 4096, 1, 0) == EINVAL
    assert lib.sal_cache_fork(r, 4096, 4096, 5, 4096, 4096, 0) == EINVAL  # more entries than sequences
    assert lib.sal_cache_fork(r, 0, 4096, 1, 4096, 4096, 0) == EINVAL
    assert lib.sal_cache_fork(r, 4096, 4096, 1, 0, 4096, 0) == EINVAL
    assert lib.sal_cache_fork(r, 4096, 4096, 1, 4096, 4098, 0) == EINVAL
    assert lib.sal_cache_resize(r, 4096, 4096, -1, None, 4096, 4096, 0) == EINVAL
    assert lib.sal_cache_resize(r, 4096, 0, 1, None, 4096, 4096, 0) == EINVAL
    assert lib.sal_cache_resize(r, 4096, 4096, 1, _window(api, sinks=-1), 4096, 4096, 0) == EINVAL
    assert lib.sal_cache_compact(r, 4096, 0, 0) == EINVAL
    for change, want in ((dict(workspace=0), EINVAL), (dict(workspace=4096 + 128), EINVAL),
                         (dict(workspace_bytes=lib.sal_cache_workspace_bytes(64, 4) - 1), EWORKSPACE)):
        b = _cache(api, **change)
        assert lib.sal_cache_resize(ctypes.byref(b), 4096, 4096, 1, None, 4096, 4096, 0) == want
        assert lib.sal_cache_compact(ctypes.byref(b), 4096, 4096, 0) == want


def test_cache_workspace_bytes(api):
    f = api.lib().sal_cache_workspace_bytes
    assert f(0, 4) == 0 and f(64, 0) == 0 and f(-1, 4) == 0
    # a counter, a pair and a page number per page, an offset per sequence
    assert f(64, 4) >= 64 * 12 + 4 * 4 and f(64, 4) % 256 == 0
    assert f(524288, 32768) >= 524288 * 12 + 32768 * 4


def test_paged_attention_refusals(api):
    lib, c = api.lib(), _cache(api)
    r = ctypes.byref(c)
    n = lib.sal_attention_paged_workspace_bytes(r, 2, 4)
    assert n > 0 and lib.sal_attention_paged_workspace_bytes(r, 0, 4) == 0
    base = dict(q=4096, row=512, head=128, batch=2, heads=4, layer=0, seqs=0, sinks=0, o=4096, ws=4096, bytes=n)

    def call(**change):
        a = {**base, **change}
        return lib.sal_attention_paged(a["q"], a["row"], a["head"], a["batch"], a["heads"], r, a["layer"], a["seqs"],
                                       _window(api, sinks=a["sinks"]), a["o"], a["ws"], a["bytes"], 0)

    assert call(batch=0) == OK and call(heads=0) == OK
    for bad in (dict(batch=-1), dict(heads=-2), dict(layer=2), dict(layer=-1), dict(row=-8), dict(head=4),
                dict(row=260), dict(sinks=-1), dict(heads=3), dict(batch=5), dict(q=0), dict(q=4104), dict(o=0),
                dict(o=4104), dict(seqs=4098), dict(ws=0), dict(ws=4096 + 16)):
        assert call(**bad) == EINVAL, bad
    assert call(batch=65536, seqs=4096) == ESHAPE and call(heads=65536) == ESHAPE
    assert call(bytes=n - 1) == EWORKSPACE


def test_stream_refusals(api):
    """The live-stream encoder: the encoder's own checks, and a cache of its heads and layers."""
    lib = api.lib()
    layers = (api.sal_layer * 2)(*[api.sal_layer(*[4096] * len(api.LAYER_FIELDS)) for _ in range(2)])
    w = api.sal_weights(4096, 4096, layers, 2, 4096, 4096)
    good = dict(kv_heads=10, head_dim=128, layers=2)
    n1, n8 = lib.sal_stream_workspace_bytes(3, 1), lib.sal_stream_workspace_bytes(3, 8)
    assert lib.sal_stream_workspace_bytes(0, 8) == 0 and lib.sal_stream_workspace_bytes(3, 0) == 0
    assert n8 >= 24 * 1280 * 2 * 5 and n1 >= 3 * (1280 * 2 * 5 + 3840 * 4)

    def both(cache=None, x=4096, batch=3, T=8, n=2, sinks=0, emb=4096, ws=4096, b1=n1, b8=n8, seqs=0, weights=w, lens=0):
        c = _cache(api, **(good if cache is None else cache))
        r, wr, win = ctypes.byref(c), ctypes.byref(weights), _window(api, left=5, sinks=sinks)
        return (lib.sal_stream_prefill(x, batch, T, lens, wr, n, win, r, seqs, emb, ws, b8, 0),
                lib.sal_stream_step(x, batch, wr, n, win, r, seqs, emb, ws, b1, 0))

    for change, want in ((dict(batch=-1), EINVAL), (dict(n=-1), EINVAL), (dict(n=3), EINVAL), (dict(sinks=-1), EINVAL),
                         (dict(x=0), EINVAL), (dict(x=4104), EINVAL), (dict(emb=0), EINVAL), (dict(ws=0), EINVAL),
                         (dict(ws=4096 + 64), EINVAL), (dict(seqs=4098), EINVAL), (dict(batch=5), EINVAL),
                         (dict(batch=6554, seqs=4096), ESHAPE), (dict(batch=0), OK), (dict(b1=n1 - 1, b8=n8 - 1), EWORKSPACE),
                         (dict(cache=dict(good, kv_heads=2)), ESHAPE), (dict(cache=dict(good, head_dim=64)), ESHAPE),
                         (dict(cache=dict(good, layers=1)), ESHAPE), (dict(cache=dict(good, page_size=24)), ESHAPE)):
        assert both(**change) == (want, want), change
    assert both(T=45001)[0] == ESHAPE and both(T=-1)[0] == EINVAL and both(T=0)[0] == OK and both(lens=4098)[0] == EINVAL
    layers[1].w_o = 0
    assert both() == (EINVAL, EINVAL)


# ----------------------------------------------------------------- the model of the tables


def test_model_grow_cut_and_free():
    m = CacheModel(pages=6, page=4, sequences=3, max_pages=4)
    m.resize([1, 0], [5, 3])
    assert m.table == [[2, -1, -1, -1], [0, 1, -1, -1], [-1] * 4] and m.lengths == [3, 5, 0]
    m.resize([1], [4])          # page 1 is free again
    m.resize([2, 0], [8, 5])    # 2 takes 1 and 3, 0 takes 4
    assert m.table == [[2, 4, -1, -1], [0, -1, -1, -1], [1, 3, -1, -1]]
    m.resize([1], [16])         # three more pages: only page 5 is free
    assert m.status == m.NO_PAGES and m.lengths == [5, 4, 8] and m.table[1] == [0, -1, -1, -1]
    m.resize([0, 0], [1, 2])
    assert m.status == m.NO_PAGES | m.BAD_LIST and m.lengths == [5, 4, 8]


def test_model_fork_shares_and_growth_copies():
    m = CacheModel(pages=8, page=4, sequences=3, max_pages=3)
    m.resize([0], [6])
    m.append([["a", "b", "c", "d", "e", "f"]], [0])
    m.fork([0, 0], [1, 2])
    assert m.table == [[0, 1, -1]] * 3
    m.resize([2, 1], [7, 6])    # only 2 grows: it gets a copy of page 1
    assert m.table == [[0, 1, -1], [0, 1, -1], [0, 2, -1]] and m.data[2][:2] == ["e", "f"]
    m.resize([0, 1], [7, 7])    # both still share page 1, so both get copies and page 1 is free
    assert m.table == [[0, 3, -1], [0, 4, -1], [0, 2, -1]]
    m.fork([1, 0], [0, 1])      # a permutation
    assert m.table[:2] == [[0, 4, -1], [0, 3, -1]]


def test_model_window_lets_pages_go_and_compacts():
    m = CacheModel(pages=9, page=4, sequences=2, max_pages=6)
    m.resize([0], [20])
    m.resize([1], [4])
    m.resize([0], [21], left=6, sinks=3)  # positions from 20 on see 14 ..: entries 1 and 2 go
    assert m.table[0] == [0, -1, -1, 3, 4, 1] and m.table[1][0] == 5
    m.compact()
    assert m.table[0] == [0, -1, -1, 3, 4, 1] and m.table[1][0] == 2
