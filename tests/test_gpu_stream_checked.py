"""The live-stream calls through both builds of the library (the bounds-checked one must refuse
no access and give the same bytes), between guard bands, and with a wait that gives up.

As in the tests of the other calls: every buffer that a call writes lies between 4 KiB of
guard bytes which stay as they were, in the normal and in the checked build; and the test hook
that withholds key tiles makes the windowed kernel's bounded waits run out, after which it winds
down, the status says so, and the next call is right.
"""
import ctypes
import time

import pytest
import torch

from gpu_util import weights
from stream_ref import attention_bound, window_reference

pytestmark = pytest.mark.gpu

GUARD, PATTERN = 4096, 0xA5
SAL_ETIMEOUT, DEFAULT_LIMIT_NS = 5, 4_000_000_000


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Guards:
    """Tensors carved out of larger allocations of guard bytes."""

    def __init__(self):
        self.all = []

    def put(self, t: torch.Tensor) -> torch.Tensor:
        n = t.numel() * t.element_size()
        raw = torch.full((GUARD + n + GUARD,), PATTERN, dtype=torch.uint8, device="cuda")
        self.all.append((raw, n))
        v = raw[GUARD:GUARD + n].view(t.dtype).view(t.shape)
        v.copy_(t)
        return v

    def intact(self) -> bool:
        return all(bool((raw[:GUARD] == PATTERN).all()) and bool((raw[GUARD + n:] == PATTERN).all())
                   for raw, n in self.all)


def _both(run):
    """run(guards) -> tensors, through the normal and the checked build: equal bytes, no refused
    access, guards intact."""
    api = _api()
    outs = []
    for checked in (False, True):
        g = Guards()
        if checked:
            with api.checked_library():
                api.check_report()
                got = [t.clone() for t in run(g)]
                rep = api.check_report()
            assert rep["count"] == 0, rep
        else:
            got = [t.clone() for t in run(g)]
        torch.cuda.synchronize()
        assert g.intact()
        outs.append(got)
    for i, (a, b) in enumerate(zip(*outs)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


@pytest.mark.parametrize("B,T,H,kvh,d,left,right,sinks,lens,offset", [
    (2, 300, 10, 10, 128, 50, 0, 4, [300, 77], 0), (3, 1000, 4, 2, 128, 130, 20, 0, None, 8),
    (2, 513, 6, 6, 64, -1, -1, 0, [129, 513], 0), (1, 129, 2, 2, 64, 0, 0, 200, None, 8), (2, 1, 3, 3, 128, -1, 0, 1, [0, 1], 8)])
def test_window(B, T, H, kvh, d, left, right, sinks, lens, offset):
    """offset: outputs 16 but not 32 bytes past an aligned address (narrower stores)."""
    g0 = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(B, h, T, d, generator=g0, device="cuda").bfloat16() for h in (H, kvh, kvh))

    def run(g):
        out = g.put(torch.zeros(B * T * H * d + 8, dtype=torch.bfloat16, device="cuda"))
        o = out[offset:offset + B * T * H * d].view(B * T, H * d)
        _api().sal_attention_window(q, k, v, left, right, sinks, None if lens is None else _ints(lens), o)
        return [out]

    _both(run)


@pytest.mark.parametrize("lengths,H,kvh,d,page,left,sinks", [
    ([1, 0, 40], 10, 10, 128, 16, -1, 0), ([700, 3, 90], 32, 2, 128, 8, 100, 5), ([3000, 1], 4, 4, 64, 64, -1, 0),
    ([500] * 40, 10, 10, 128, 16, 200, 3), ([9000, 8000], 20, 1, 128, 256, -1, 0)])
def test_paged_attention(lengths, H, kvh, d, page, left, sinks):
    api = _api()
    g0 = torch.Generator(device="cuda").manual_seed(page)
    counts = [-(-n // page) for n in lengths]
    pool, width = sum(counts) + 1, max(counts) + 1
    order = torch.randperm(pool, generator=g0, device="cuda").tolist()
    table, at = [], 0
    for c in counts:
        table.append(order[at:at + c] + [-1] * (width - c))
        at += c
    k, v = (torch.randn(1, pool, kvh, page, d, generator=g0, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(len(lengths), H, d, generator=g0, device="cuda").bfloat16()

    def run(g):
        cache = api.PagedCache(k, v, _ints(table), _ints(lengths))
        o = g.put(torch.zeros(len(lengths), H * d, dtype=torch.bfloat16, device="cuda"))
        ws = g.put(api.attention_paged_workspace(cache, len(lengths), H))
        for _ in range(2):  # the second on the scratch that the first left
            api.sal_attention_paged(q, cache, left, sinks, out=o, workspace=ws)
        return [o]

    _both(run)


@pytest.mark.parametrize("page,pages,sequences,max_pages", [(8, 70, 5, 20), (32, 33, 40, 3)])
def test_cache(page, pages, sequences, max_pages):
    api = _api()
    g0 = torch.Generator(device="cuda").manual_seed(page)
    shape = (2, pages, 3, page, 64)
    k0, v0 = (torch.randn(shape, generator=g0, device="cuda").bfloat16() for _ in range(2))
    new = torch.randn(sequences, 3, 2 * page, 64, generator=g0, device="cuda").bfloat16()

    def run(g):
        def tables():
            return (g.put(torch.full((sequences, max_pages), -1, dtype=torch.int32, device="cuda")),
                    g.put(torch.zeros(sequences, dtype=torch.int32, device="cuda")))
        k, v = g.put(k0), g.put(v0)
        n = api.lib().sal_cache_workspace_bytes(pages, sequences)
        ws = g.put(torch.zeros(n, dtype=torch.uint8, device="cuda"))
        status = g.put(torch.zeros(1, dtype=torch.int32, device="cuda"))
        a = api.PagedCache(k, v, *tables(), status, ws)
        b = a.with_tables(*tables())
        every = list(range(sequences))
        api.sal_cache_resize(a, _ints(every), _ints([(7 * s) % (page * max_pages // 4 + 1) for s in every]))
        api.sal_cache_append(a, new, new, _ints([s % 3 for s in every]), layer=1)
        api.sal_cache_fork(a, _ints([0, 1]), _ints([2, 3]), out=b)
        api.sal_cache_resize(b, _ints([3, 0]), _ints([page + 1, 2]), left=3, sinks=1)
        api.sal_cache_resize(b, _ints([1]), _ints([page * max_pages]), out=a)
        api.sal_cache_resize(b, _ints([1, 1]), _ints([0, 0]))
        api.sal_cache_copy_pages(b, _ints([0, 1, pages]), _ints([pages - 1, pages - 2, 0]))
        api.sal_cache_compact(b, out=a)
        api.sal_cache_compact(a)
        return [k, v, a.table, a.lengths, b.table, b.lengths, status]

    _both(run)


def test_streams():
    """2,000 positions (the residual products split K below 1,793 rows, whose partial sums land in no
    fixed order) and steps of one layer's worth of rows; steps are compared by their cache only."""
    api = _api()
    _, _, dw = weights(2)
    x0 = torch.randn(1, 2000, 1280, device="cuda")

    def run(g):
        cache = api.PagedCache.empty(2, 140, 10, 16, 128, 1, 130)
        cache.k.zero_(), cache.v.zero_()
        api.sal_cache_resize(cache, _ints([0]), _ints([2000]))
        x = g.put(x0)
        emb = g.put(torch.zeros(1, 2000, 1280, dtype=torch.bfloat16, device="cuda"))
        ws = g.put(api.stream_workspace(1, 2000))
        api.sal_stream_prefill(x, dw, 2, cache, 100, 4, emb=emb, workspace=ws)
        api.sal_cache_resize(cache, _ints([0]), _ints([2001]))
        y = g.put(x0[:, 5].clone())
        e = g.put(torch.zeros(1, 1280, dtype=torch.bfloat16, device="cuda"))
        w1 = g.put(api.stream_workspace(1))
        before = [cache.k.clone(), cache.v.clone()]
        api.sal_stream_step(y, dw, 2, cache, 100, 4, emb=e, workspace=w1)
        return [x, emb, *before, cache.k[0], cache.v[0]]  # (layer 0's new row comes before any residual product)

    _both(run)


@pytest.mark.parametrize("d,heads", [(128, 10), (64, 16)])
@pytest.mark.parametrize("tile", [0, 1, 3])
def test_withheld_tiles_time_out_and_the_next_call_is_right(d, heads, tile):
    api = _api()
    T = 3000
    q, k, v = (torch.randn(1, heads, T, d, device="cuda").bfloat16() for _ in range(3))
    assert api.sal_last_device_status() == 0
    api.sal_set_wait_limit_ns(20_000_000)
    try:
        t0 = time.perf_counter()
        api.sal_attention_window_withhold(q, k, v, tile, 700, 0, 4)
        status = api.sal_last_device_status()
        elapsed = time.perf_counter() - t0
    finally:
        api.sal_set_wait_limit_ns(DEFAULT_LIMIT_NS)
    assert status == SAL_ETIMEOUT and elapsed < 2.0, elapsed
    assert api.sal_last_device_status() == 0
    o = api.sal_attention_window(q, k, v, 700, 0, 4)
    assert api.sal_last_device_status() == 0
    ref, spread = window_reference(q, k, v, 700, 0, 4, [T])
    off = (o.double().reshape(ref.shape) - ref).abs() - attention_bound(ref, spread)
    assert float(off.max()) <= 0


def test_withholding_past_the_last_tile_changes_nothing():
    api = _api()
    q, k, v = (torch.randn(2, 4, 500, 128, device="cuda").bfloat16() for _ in range(3))
    a = api.sal_attention_window_withhold(q, k, v, 100, 90, 5, 2)
    assert api.sal_last_device_status() == 0
    assert torch.equal(a, api.sal_attention_window(q, k, v, 90, 5, 2))
