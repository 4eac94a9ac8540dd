"""sal_attention_window against the 64-bit form of its mask (stream_ref): clips of one to a
few thousand positions, windows that end inside, at and past a 128-row tile, grouped heads,
lengths, what lies past them, other streams, captured graphs, offsets past 32 bits."""
import pytest
import torch

from stream_ref import attention_bound, visible, window_reference

pytestmark = pytest.mark.gpu


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def _inputs(B, T, H, kvh, d, seed=0, q_scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + H)
    return (_randn(g, B, H, T, d) * q_scale), _randn(g, B, kvh, T, d), _randn(g, B, kvh, T, d)


def _compare(o, q, k, v, left, right, sinks, lengths=None, q_scale=1.0):
    B, H, T, d = q.shape
    lens = [T] * B if lengths is None else lengths
    ref, spread = window_reference(q, k, v, left, right, sinks, lens)
    got = o.double().reshape(B, T, H, d)
    for b, n in enumerate(lens):
        n = max(0, min(T, n))
        off = (got[b, :n] - ref[b, :n]).abs() - attention_bound(ref[b, :n], spread[b, :n], q_scale)
        assert n == 0 or float(off.max()) <= 0, (b, float(off.max()))


CASES = [
    # batch, T, heads, kv_heads, head_dim, left, right, sinks
    (1, 1, 10, 10, 128, -1, 0, 0), (1, 1, 2, 1, 64, 0, 0, 5), (2, 7, 10, 10, 128, 2, 0, 1), (1, 127, 4, 4, 64, -1, -1, 0),
    (1, 128, 4, 2, 128, 50, 50, 0), (3, 129, 4, 4, 128, 128, 0, 0), (1, 129, 2, 2, 64, 127, 1, 3),
    (1, 300, 10, 10, 128, -1, 0, 0), (2, 374, 10, 10, 128, 50, 50, 4), (1, 383, 3, 1, 64, 0, -1, 0),
    (1, 640, 2, 2, 128, 0, 0, 130), (1, 640, 2, 2, 64, 100, 0, 128), (1, 777, 5, 5, 128, 256, 128, 0),
    (1, 777, 6, 2, 64, 255, 300, 129), (2, 1000, 2, 2, 128, 375, 0, 8), (1, 1500, 3, 3, 128, 700, 0, 640),
    (1, 1025, 32, 2, 128, 100, 0, 4), (1, 513, 10, 2, 128, -1, -1, 0), (1, 2049, 1, 1, 64, 1, 513, 1),
    (1, 900, 3, 3, 128, 5000, 5000, 5000), (1, 400, 2, 2, 128, 1 << 40, 0, 1 << 40),
    (5, 257, 7, 7, 64, 64, 64, 2), (17, 150, 10, 10, 128, 20, 0, 1),
]


@pytest.mark.parametrize("case", CASES)
def test_matches_the_mask(case):
    B, T, H, kvh, d, left, right, sinks = case
    q, k, v = _inputs(B, T, H, kvh, d)
    o = _api().sal_attention_window(q, k, v, left=left, right=right, sinks=sinks)
    _compare(o, q, k, v, left, right, sinks)


@pytest.mark.parametrize("T,H,kvh,d,left,right,sinks", [
    (300, 10, 10, 128, 50, 0, 4), (300, 4, 2, 64, -1, -1, 0), (700, 4, 4, 128, 130, 20, 0), (130, 3, 3, 128, 0, 0, 200)])
def test_lengths_and_what_lies_past_them(T, H, kvh, d, left, right, sinks):
    """Clips of 0, 1, some, all and (clamped) more or less than all positions; NaN and infinities
    past each length change nothing, and the rows past it stay as they were."""
    lens = [0, 1, T // 2, 127, 128, 129, T, T + 50, -3]
    B = len(lens)
    q, k, v = _inputs(B, T, H, kvh, d, seed=1)
    clean = [x.clone() for x in (q, k, v)]
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        for b, n in enumerate(lens):
            x[b, :, max(0, min(n, T)):] = bad
    o = torch.full((B * T, H * d), 7.0, dtype=torch.bfloat16, device="cuda")
    api = _api()
    api.sal_attention_window(q, k, v, left=left, right=right, sinks=sinks,
                             lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), out=o)
    _compare(o, *clean, left, right, sinks, lens)
    rows = o.reshape(B, T, H * d)
    for b, n in enumerate(lens):
        assert bool((rows[b, max(0, min(n, T)):] == 7.0).all()), b
    # what lies past the lengths is not used: other padding, the same bits
    again = torch.full_like(o, 7.0)
    api.sal_attention_window(*clean, left=left, right=right, sinks=sinks,
                             lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), out=again)
    assert torch.equal(o, again)
    # and a clip alone, whose keys may fall into other tiles, agrees within the bound
    for b in (3, 4, 5):
        alone = [x[b:b + 1, :, :lens[b]].contiguous() for x in clean]
        _compare(api.sal_attention_window(*alone, left=left, right=right, sinks=sinks), *alone, left, right, sinks)


@pytest.mark.parametrize("B,T,H,kvh,d", [(33, 300, 2, 2, 128), (70, 257, 4, 2, 64), (64, 129, 3, 3, 64),
                                         (100, 40, 4, 4, 128), (2, 4000, 10, 10, 128)])
@pytest.mark.parametrize("which", ["ragged", "one", "none"])
def test_many_clips_of_different_lengths(B, T, H, kvh, d, which):
    """The list of items that lengths reach: more clips than a warp has lanes, most of them short,
    one alone, none at all."""
    g = torch.Generator().manual_seed(B + T)
    lens = torch.randint(0, T + 1, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.4] = 0
    lens[B // 2] = T
    if which != "ragged":
        lens[torch.arange(B) != B // 2] = 0
    if which == "none":
        lens[:] = 0
    lens = lens.tolist()
    q, k, v = _inputs(B, T, H, kvh, d, seed=13)
    o = torch.full((B * T, H * d), 7.0, dtype=torch.bfloat16, device="cuda")
    _api().sal_attention_window(q, k, v, left=90, right=5, sinks=2,
                                lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), out=o)
    _compare(o, q, k, v, 90, 5, 2, lens)
    rows = o.reshape(B, T, H * d)
    assert all(bool((rows[b, n:] == 7.0).all()) for b, n in enumerate(lens))


@pytest.mark.parametrize("T,H,kvh,d,left,right,sinks", [
    (300, 2, 2, 128, 20, 0, 4), (300, 4, 2, 64, 40, 10, 0), (1500, 10, 10, 128, 100, 0, 200), (3000, 16, 16, 64, 33, 65, 3),
    (2100, 8, 2, 128, 150, 0, 4), (200, 3, 3, 128, -1, 0, 0)])
def test_values_that_are_no_numbers(T, H, kvh, d, left, right, sinks):
    """Keys and values that are infinite or NaN reach the rows that see them, and no other row of
    their tiles."""
    q, k, v = _inputs(2, T, H, kvh, d, seed=11)
    wrong = torch.zeros(T, dtype=torch.bool)
    for at, (x, bad) in zip((T // 7, T // 2, T // 2 + 70, T - 5),
                            ((v, float("nan")), (v, float("-inf")), (k, float("nan")), (v, float("inf")))):
        x[0, :, at] = bad
        wrong[at] = True
    o = _api().sal_attention_window(q, k, v, left=left, right=right, sinks=sinks).double().reshape(2, T, H, d)
    p = torch.arange(T)[:, None]
    hit = (visible(p, torch.arange(T)[None, :], T, left, right, sinks) & wrong[None, :]).any(1).cuda()
    assert 0 < int(hit.sum()) < T
    ref, spread = window_reference(q, k, v, left, right, sinks, [T, T])
    off = (o - ref).abs() - attention_bound(ref, spread)
    assert bool((off[0, ~hit] <= 0).all()) and bool((off[1] <= 0).all())
    assert not bool(torch.isfinite(o[0, hit]).any())


@pytest.mark.parametrize("d", [64, 128])
def test_each_position_alone_returns_its_value(d):
    """left = right = 0 without sinks: every position sees itself only, so o = v to the bit."""
    q, k, v = _inputs(2, 1111, 3, 3, d, seed=2)
    o = _api().sal_attention_window(q, k, v, left=0, right=0)
    assert torch.equal(o.reshape(2, 1111, 3, d).transpose(1, 2), v)


def test_scores_that_one_key_takes():
    """Queries eight times as long: most rows' weight sits on a key or two."""
    q, k, v = _inputs(1, 600, 4, 4, 128, seed=3, q_scale=8.0)
    o = _api().sal_attention_window(q, k, v, left=200, right=10, sinks=3)
    _compare(o, q, k, v, 200, 10, 3, q_scale=8.0)


def test_scores_that_rise_along_the_keys():
    """Every key tile brings a new maximum (the running maximum is replaced again and again)."""
    q, k, v = _inputs(1, 1300, 2, 2, 128, seed=4)
    ramp = torch.linspace(0.0, 6.0, 1300, device="cuda")[:, None]
    q = torch.ones_like(q) * 0.5
    k = (k * 0.05 + ramp).bfloat16()
    for left, right in ((-1, 0), (-1, -1), (300, 0)):
        o = _api().sal_attention_window(q, k, v, left=left, right=right, sinks=2)
        # sum |q_i k_i| is up to 128 * 0.5 * 6 here: three times the bound's unit
        _compare(o, q, k, v, left, right, 2, q_scale=3.0)


def test_without_limits_it_is_the_full_attention():
    """The same function as sal_attention_heads: both are within the bound of each other."""
    api = _api()
    for H, d in ((10, 128), (16, 64)):
        q, k, v = _inputs(2, 500, H, H, d, seed=5)
        o = api.sal_attention_window(q, k, v)
        _compare(o, q, k, v, -1, -1, 0)
        full = api.sal_attention_heads(q, k, v).reshape(o.shape)
        assert float((o.double() - full.double()).norm() / full.double().norm()) < 2 * 2.0 ** -8


def test_repeated_calls_agree_to_the_bit():
    q, k, v = _inputs(2, 1500, 10, 10, 128, seed=6)
    api = _api()
    first = api.sal_attention_window(q, k, v, left=300, right=5, sinks=4).clone()
    for _ in range(3):
        assert torch.equal(api.sal_attention_window(q, k, v, left=300, right=5, sinks=4), first)


def test_other_stream_and_captured_graph():
    api = _api()
    q, k, v = _inputs(2, 700, 10, 10, 128, seed=8)
    lens = torch.tensor([700, 333], dtype=torch.int32, device="cuda")
    want = api.sal_attention_window(q, k, v, left=100, right=0, sinks=4, lengths=lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(want)
    with torch.cuda.stream(side):
        api.sal_attention_window(q, k, v, left=100, right=0, sinks=4, lengths=lens, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        api.sal_attention_window(q, k, v, left=100, right=0, sinks=4, lengths=lens, out=out)
    q2, k2, v2 = _inputs(2, 700, 10, 10, 128, seed=9)
    lens2 = torch.tensor([12, 700], dtype=torch.int32, device="cuda")
    want2 = api.sal_attention_window(q2, k2, v2, left=100, right=0, sinks=4, lengths=lens2)
    for a, b in ((q, q2), (k, k2), (v, v2), (lens, lens2)):
        a.copy_(b)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


def test_offsets_past_32_bits():
    """2.6 G elements per tensor: the last clip's rows lie past 2^32 bytes and 2^31 elements."""
    B, T, H, d = 32, 64000, 10, 128
    q = torch.zeros(B, H, T, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(q)
    g = torch.Generator(device="cuda").manual_seed(1)
    for b in (0, B - 1):
        v[b] = _randn(g, H, T, d)
    o = torch.zeros(B * T, H * d, dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[0], lens[B - 1] = 100, T
    _api().sal_attention_window(q, q, v, left=0, right=0, lengths=lens, out=o)
    rows = o.reshape(B, T, H, d)
    assert torch.equal(rows[B - 1].transpose(0, 1), v[B - 1])
    assert torch.equal(rows[0, :100].transpose(0, 1), v[0, :, :100])
    assert not bool(rows[1:B - 1].any()) and not bool(rows[0, 100:].any())


def test_python_refusals():
    api = _api()
    q, k, v = _inputs(1, 32, 4, 2, 64, seed=10)
    for bad in (dict(k=k[:, :, :16].contiguous()), dict(v=v.float()), dict(q=q.transpose(1, 2)), dict(k=k.cpu()),
                dict(lengths=torch.zeros(1, dtype=torch.int64, device="cuda")),
                dict(lengths=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(out=torch.empty(32, 255, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            api.sal_attention_window(**{**dict(q=q, k=k, v=v), **bad})
    with pytest.raises(api.SalError):
        api.sal_attention_window(q, k, v, sinks=-1)
    with pytest.raises(api.SalError):
        api.sal_attention_window(q[:, :3].contiguous(), k, v)
