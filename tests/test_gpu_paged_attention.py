"""sal_attention_paged against the 64-bit form (stream_ref), and a run of the live-stream
calls together: positions appended one by one, sequences forked, pages let go and compacted
between, every step's attention equal to the windowed attention over the same positions."""
import pytest
import torch

from stream_ref import attention_bound, paged_reference

pytestmark = pytest.mark.gpu


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _make(lengths, H, kvh, d, page, seed=0, q_scale=1.0, spare=3, max_pages=None):
    """A cache whose unused slots hold NaN, its pages handed out in random order."""
    g = torch.Generator(device="cuda").manual_seed(seed + H + page)
    counts = [-(-n // page) for n in lengths]
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    max_pages = max_pages or max(1, max(counts) + 1)
    shape = (2, pages, kvh, page, d)
    k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full(shape, float("inf"), dtype=torch.bfloat16, device="cuda")
    table, at = [], 0
    for n, c in zip(lengths, counts):
        rows = order[at:at + c]
        at += c
        table.append(rows + [-1] * (max_pages - c))
        for i, p in enumerate(rows):
            top = min(page, n - i * page)
            k[:, p, :, :top] = torch.randn(2, kvh, top, d, generator=g, device="cuda").bfloat16()
            v[:, p, :, :top] = torch.randn(2, kvh, top, d, generator=g, device="cuda").bfloat16()
    q = (torch.randn(len(lengths), H, d, generator=g, device="cuda") * q_scale).bfloat16()
    return _api().PagedCache(k, v, _ints(table), _ints(lengths)), q


def _compare(o, q, cache, layer, left, sinks, seqs=None, q_scale=1.0):
    ref, spread = paged_reference(q, cache.k[layer], cache.v[layer], cache.table, cache.lengths, left, sinks, seqs)
    off = (o.double().reshape(ref.shape) - ref).abs() - attention_bound(ref, spread, q_scale)
    assert float(off.max()) <= 0, float(off.max())


CASES = [
    # lengths, heads, kv_heads, head_dim, page, left, sinks
    ([1], 10, 10, 128, 16, -1, 0), ([0, 1, 2], 10, 10, 128, 16, -1, 0), ([15, 16, 17, 31, 32, 33], 4, 4, 64, 16, -1, 0),
    ([7, 8, 9, 100], 4, 2, 128, 8, -1, 0), ([255, 256, 257, 513], 2, 1, 64, 256, -1, 0), ([750], 10, 10, 128, 16, -1, 0),
    ([750, 3, 400], 10, 10, 128, 16, 100, 0), ([750, 3, 400], 10, 10, 128, 16, 100, 5), ([700], 32, 2, 128, 64, -1, 0),
    ([700, 50], 32, 2, 128, 64, 33, 40), ([300], 20, 1, 64, 32, -1, 0), ([300, 299], 40, 1, 128, 32, 0, 1),
    ([3000], 12, 4, 64, 8, -1, 0), ([5000, 1], 8, 4, 128, 128, -1, 0), ([1000], 10, 2, 128, 16, 0, 0),
    ([1000, 40], 10, 2, 128, 16, 15, 17), ([600] * 40, 10, 10, 128, 16, -1, 0), ([90] * 200, 4, 4, 64, 16, 50, 2),
    ([2000], 2, 2, 128, 16, 1 << 40, 1 << 40), ([500], 2, 2, 64, 8, 100, 390), ([500], 2, 2, 64, 8, 100, 700),
]


@pytest.mark.parametrize("case", CASES)
def test_matches_the_visible_keys(case):
    lengths, H, kvh, d, page, left, sinks = case
    cache, q = _make(lengths, H, kvh, d, page)
    for layer in (0, 1):
        o = _api().sal_attention_paged(q, cache, left, sinks, layer)
        _compare(o, q, cache, layer, left, sinks)


def test_pages_let_go_bad_entries_and_lengths():
    """Entries of -1 and out of range hide their keys wherever they stand; lengths below 0 and
    past the table are clamped."""
    cache, q = _make([200, 200, 200, 64, 30], 4, 2, 128, 16, seed=1)
    cache.table[0, 3:8] = -1
    cache.table[1, 0] = cache.k.shape[1]
    cache.table[1, 12] = -2 ** 31
    cache.table[2, :] = -1
    cache.lengths[3] = 100000   # the entries past its four pages are -1
    cache.lengths[4] = -5
    o = _api().sal_attention_paged(q, cache)
    _compare(o, q, cache, 0, -1, 0)
    assert not bool(o[2].any()) and not bool(o[4].any())
    o = _api().sal_attention_paged(q, cache, left=90, sinks=20)
    _compare(o, q, cache, 0, 90, 20)


@pytest.mark.parametrize("H,kvh,d,page,left,sinks", [(10, 10, 128, 16, 100, 5), (16, 2, 64, 8, 37, 0), (4, 4, 128, 64, 0, 17)])
def test_hidden_keys_and_values_that_are_no_numbers(H, kvh, d, page, left, sinks):
    """Positions between the first ones and the window hold NaN and infinities, up to the visible
    ones' edges: nothing of it reaches a result."""
    lengths = [150, 333, 1000, 2 + left, left + sinks + 9]
    cache, q = _make(lengths, H, kvh, d, page, seed=12)
    clean = _api().sal_attention_paged(q, cache, left, sinks, 1)
    for s, n in enumerate(lengths):
        for j in range(sinks, n - 1 - left):
            at = int(cache.table[s, j // page])
            cache.k[:, at, :, j % page] = float("inf")
            cache.v[:, at, :, j % page] = float("nan") if j % 2 else float("-inf")
    assert torch.equal(_api().sal_attention_paged(q, cache, left, sinks, 1), clean)
    _compare(clean, q, cache, 1, left, sinks)


def test_rows_name_their_sequences():
    """Rows in another order, one sequence twice, sequences out of range (zeros)."""
    cache, _ = _make([40, 0, 333, 100], 10, 10, 128, 16, seed=2)
    seqs = [2, 0, 2, 3, -1, 4, 1, 2 ** 31 - 1]
    q = torch.randn(len(seqs), 10, 128, device="cuda").bfloat16()
    o = _api().sal_attention_paged(q, cache, seqs=_ints(seqs))
    _compare(o, q, cache, 0, -1, 0, seqs)
    for b in (4, 5, 6, 7):
        assert not bool(o[b].any())


def test_query_strides():
    """Queries laid out [heads, batch, head_dim], and rows with other data between them."""
    cache, q = _make([100, 200, 300], 10, 10, 128, 16, seed=3)
    api = _api()
    want = api.sal_attention_paged(q, cache)
    across = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert across.stride(0) == 128 and torch.equal(api.sal_attention_paged(across, cache), want)
    wide = torch.full((3, 30, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 10:20] = q
    assert torch.equal(api.sal_attention_paged(wide[:, 10:20], cache), want)


def test_scores_that_one_key_takes():
    cache, q = _make([900, 64], 10, 10, 128, 16, seed=4, q_scale=8.0)
    o = _api().sal_attention_paged(q, cache)
    _compare(o, q, cache, 0, -1, 0, q_scale=8.0)


def test_repeated_calls_agree_to_the_bit():
    cache, q = _make([5000, 77, 2300], 32, 2, 128, 16, seed=5)
    api = _api()
    first = api.sal_attention_paged(q, cache).clone()
    for _ in range(4):
        assert torch.equal(api.sal_attention_paged(q, cache), first)


def test_other_streams_with_workspaces_of_their_own():
    """Two calls that may overlap, each with its workspace."""
    api = _api()
    cache, q = _make([9000, 8000], 32, 2, 128, 64, seed=6)
    q2 = torch.randn_like(q)
    want, want2 = api.sal_attention_paged(q, cache), api.sal_attention_paged(q2, cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in range(2)]
    spaces = [api.attention_paged_workspace(cache, 2, 32) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, o, w in zip(streams, (q, q2), outs, spaces):
            api.sal_attention_paged(x, cache, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want2)


def test_captured_and_replayed_with_other_lengths():
    """The graph follows the tables and lengths as they are at replay, and two graphs that share
    a workspace in turn do not disturb each other."""
    api = _api()
    cache, q = _make([4000, 100], 10, 10, 128, 16, seed=7)
    space = api.attention_paged_workspace(cache, 2, 10)
    outs, graphs = [], []
    for left in (-1, 300):
        out = torch.zeros(2, 1280, dtype=torch.bfloat16, device="cuda")
        api.sal_attention_paged(q, cache, left=left, out=out, workspace=space)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.sal_attention_paged(q, cache, left=left, out=out, workspace=space)
        outs.append(out)
        graphs.append(graph)
    for lens in ([4000, 100], [1, 0], [2049, 17], [3999, 99]):
        cache.lengths.copy_(_ints(lens))
        for left, out, graph in zip((-1, 300), outs, graphs):
            out.fill_(9.0)
            graph.replay()
        for left, out in zip((-1, 300), outs):
            _compare(out, q, cache, 0, left, 0)


def test_one_head_of_a_long_cache():
    """100,000 positions of one sequence, one head: the axis split as far as it goes."""
    n = 100000
    pages = n // 16 + 3
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(1, pages, 1, 16, 128, generator=g, device="cuda").bfloat16()
    v = torch.randn(1, pages, 1, 16, 128, generator=g, device="cuda").bfloat16()
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None, :n // 16 + 1].contiguous()
    cache = _api().PagedCache(k, v, table, _ints([n - 5]))
    q = torch.randn(1, 1, 128, generator=g, device="cuda").bfloat16()
    o = _api().sal_attention_paged(q, cache)
    _compare(o, q, cache, 0, -1, 0)


def test_pages_past_32_bits():
    """A pool of 2.7 G elements, the sequence's pages in its last gigabyte, in layer 1's slab."""
    pages, H, ps, hd = 66000, 10, 16, 128
    k = torch.zeros(2, pages, H, ps, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[1, -40:], v[1, -40:] = (torch.randn(40, H, ps, hd, device="cuda").bfloat16() for _ in range(2))
    table = torch.arange(pages - 40, pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    cache = _api().PagedCache(k, v, table, _ints([630]))
    q = torch.randn(1, H, hd, device="cuda").bfloat16()
    o = _api().sal_attention_paged(q, cache, layer=1)
    _compare(o, q, cache, 1, -1, 0)


def test_python_refusals():
    api = _api()
    cache, q = _make([40, 20], 4, 2, 128, 16, seed=8)
    for bad in (q[:, :, :64], q.float(), q.cpu(), q.transpose(1, 2)):
        with pytest.raises(ValueError):
            api.sal_attention_paged(bad, cache)
    with pytest.raises(ValueError):
        api.sal_attention_paged(q, cache, seqs=_ints([0]))
    with pytest.raises(api.SalError):
        api.sal_attention_paged(q[:, :3], cache)
    with pytest.raises(api.SalError):
        api.sal_attention_paged(q, cache, layer=2)
    with pytest.raises(api.SalError):
        api.sal_attention_paged(torch.cat([q, q]), cache)  # four rows, two sequences
    with pytest.raises(api.SalError):
        api.sal_attention_paged(q, cache, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("H,kvh,d,page,left,sinks", [(10, 10, 128, 16, 40, 3), (8, 2, 64, 8, -1, 0),
                                                     (4, 4, 128, 32, 20, 0)])
def test_streams_step_by_step(H, kvh, d, page, left, sinks):
    """Five live streams of a two-layer cache: a prompt of uneven lengths through the windowed
    attention, then single positions; on the way one stream forks, one ends and starts again,
    pages outside the window are let go and the pool is compacted. Every step's rows must match
    the windowed attention's last row over the stream's whole history."""
    api = _api()
    g = torch.Generator(device="cuda").manual_seed(page)
    S, layers, T = 5, 2, 70
    cache = api.PagedCache.empty(layers, 200, kvh, page, d, S, 40)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    lens = [70, 1, 33, 0, 64]
    k, v, q = rnd(layers, S, kvh, T, d), rnd(layers, S, kvh, T, d), rnd(S, H, T, d)
    every = _ints(list(range(S)))
    api.sal_cache_resize(cache, every, _ints(lens), left, sinks)
    for layer in range(layers):
        api.sal_cache_append(cache, k[layer], v[layer], _ints([0] * S), layer=layer)
    hist = [[(k[la, s, :, :n], v[la, s, :, :n]) for la in range(layers)] for s, n in enumerate(lens)]

    def check(rows, layer):
        """The cache's attention for the newest position of `rows` against the full history's."""
        x = rnd(len(rows), H, d)
        o = api.sal_attention_paged(x, cache, left, sinks, layer, _ints(rows)).reshape(len(rows), H, d)
        for i, s in enumerate(rows):
            kk, vv = hist[s][layer]
            n = kk.shape[1]
            if n == 0:
                assert not bool(o[i].any())
                continue
            qq = torch.zeros(1, H, n, d, dtype=torch.bfloat16, device="cuda")
            qq[0, :, -1] = x[i]
            want = api.sal_attention_window(qq, kk[None].contiguous(), vv[None].contiguous(), left, 0, sinks)
            spread = vv.abs().amax().double()
            # two kernels, each within the bound of the 64-bit result
            off = (o[i].double() - want[-1].double().reshape(H, d)).abs()
            assert float((off - 2 * attention_bound(o[i].double(), spread)).max()) <= 0

    check(list(range(S)), 0)
    for step in range(45):
        if step == 5:   # stream 2 goes on as 0 as well
            api.sal_cache_fork(cache, _ints([2]), _ints([0]))
            hist[0] = list(hist[2])
        if step == 11:  # stream 4 ends, and starts again with the next position
            api.sal_cache_resize(cache, _ints([4]), _ints([0]))
            hist[4] = [(kk[:, :0], vv[:, :0]) for kk, vv in hist[4]]
        if step in (17, 30):
            api.sal_cache_compact(cache)
        rows = [0, 1, 2, 4] if step % 3 else [3, 2, 0]
        old = [hist[s][0][0].shape[1] for s in rows]
        api.sal_cache_resize(cache, _ints(rows), _ints([n + 1 for n in old]), left, sinks)
        for layer in range(layers):
            nk, nv = rnd(len(rows), kvh, 1, d), rnd(len(rows), kvh, 1, d)
            api.sal_cache_append(cache, nk, nv, _ints(old), _ints(rows), layer)
            for i, s in enumerate(rows):
                kk, vv = hist[s][layer]
                hist[s][layer] = (torch.cat([kk, nk[i]], 1), torch.cat([vv, nv[i]], 1))
            check(rows, layer)
    cache.check()
    if left >= 0:  # what the window does not need has been let go
        used = int((cache.table >= 0).sum())
        assert used <= S * (2 + -(-left // page) + -(-sinks // page) + 1)
