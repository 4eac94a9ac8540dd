"""The encoder over live streams against a plain 64-bit form of its layers with the causal
window mask: a prefill of uneven lengths, single steps of all or some streams, a fork, an end and
a new start, pages let go behind the window, a captured step. Tolerance: rel-L2 below 1e-2 per
stream position block, as the encoder's own parity tests (bf16 weights, activations and P)."""
import numpy as np
import pytest
import torch

from gpu_util import rel_l2, to64, weights
from stream_ref import visible

pytestmark = pytest.mark.gpu

LAYERS, WIDTH, HEADS, HD = 2, 1280, 10, 128


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).cuda()


def _norm(x, g, b):
    m = x.mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + 1e-5) * g + b


def _reference(x, wf, left, sinks):
    """Final LayerNorm of LAYERS layers over positions 0 .. n - 1 of one stream, x [n, 1280]."""
    x, n = x.double(), x.shape[0]
    p = torch.arange(n, device="cuda")
    seen = visible(p[:, None], p[None, :], n, left, 0, sinks)
    angle = p[:, None].double() * 10000.0 ** (-torch.arange(64, device="cuda").double() / 64)
    cos, sin = torch.cos(angle), torch.sin(angle)

    def heads(y):
        return y.reshape(n, HEADS, HD).transpose(0, 1)

    def rotate(y, gain):
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * gain
        a, b = y[..., :64], y[..., 64:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    for lw in wf["layers"][:LAYERS]:
        w = {k: _t(v) for k, v in lw.items()}
        qkv = _norm(x, w["ln1_g"], w["ln1_b"]) @ w["w_qkv"].T + w["b_qkv"]
        q, k, v = (heads(qkv[:, i * WIDTH:(i + 1) * WIDTH]) for i in range(3))
        s = rotate(q, w["qn_g"]) @ rotate(k, w["kn_g"]).transpose(-1, -2) / HD ** 0.5
        o = torch.softmax(s.masked_fill(~seen, float("-inf")), -1) @ v
        x = x + o.transpose(0, 1).reshape(n, WIDTH) @ w["w_o"].T + w["b_o"]
        u = torch.nn.functional.gelu(_norm(x, w["ln2_g"], w["ln2_b"]) @ w["w1"].T + w["b1"])
        x = x + u @ w["w2"].T + w["b2"]
    return _norm(x, _t(wf["lnf_g"]), _t(wf["lnf_b"])).cpu().numpy()


@pytest.mark.parametrize("left,sinks,page", [(-1, 0, 16), (20, 0, 8), (20, 5, 16), (0, 1, 32)])
def test_prefill_and_steps(left, sinks, page):
    api = _api()
    _, wf, dw = weights(LAYERS)
    g = torch.Generator(device="cuda").manual_seed(page)
    x0 = lambda *s: torch.randn(*s, WIDTH, generator=g, device="cuda")  # noqa: E731
    S, T = 4, 150
    lens = [150, 1, 37, 129]
    cache = api.PagedCache.empty(LAYERS, 120, HEADS, page, HD, S, 40)
    every = _ints(list(range(S)))
    api.sal_cache_resize(cache, every, _ints(lens), left, sinks)
    first = x0(S, T)
    emb = api.sal_stream_prefill(first.clone(), dw, LAYERS, cache, left, sinks, _ints(lens))
    hist = [first[s, :n] for s, n in enumerate(lens)]
    want = [_reference(h, wf, left, sinks) for h in hist]
    for s, n in enumerate(lens):
        assert rel_l2(to64(emb[s, :n]), want[s]) < 1e-2, s
    for step in range(12):
        if step == 4:  # stream 1 goes on as 2
            api.sal_cache_fork(cache, _ints([2]), _ints([1]))
            hist[1] = hist[2]
        if step == 7:  # stream 3 ends and starts again
            api.sal_cache_resize(cache, _ints([3]), _ints([0]))
            hist[3] = hist[3][:0]
        if step == 9:
            api.sal_cache_compact(cache)
        rows = [3, 1, 0, 2] if step % 2 else [1, 3]
        new = x0(len(rows))
        api.sal_cache_resize(cache, _ints(rows), _ints([hist[s].shape[0] + 1 for s in rows]), left, sinks)
        emb = api.sal_stream_step(new.clone(), dw, LAYERS, cache, left, sinks, _ints(rows))
        for i, s in enumerate(rows):
            hist[s] = torch.cat([hist[s], new[i:i + 1]])
            assert rel_l2(to64(emb[i]), _reference(hist[s], wf, left, sinks)[-1]) < 1e-2, (step, s)
    cache.check()


def test_steps_equal_a_longer_prefill():
    """A prefill of 40 positions and 8 steps against a prefill of 48: the same function."""
    api = _api()
    _, _, dw = weights(LAYERS)
    x = torch.randn(2, 48, WIDTH, device="cuda")
    emb, caches = {}, {}
    for n in (40, 48):
        c = caches[n] = api.PagedCache.empty(LAYERS, 16, HEADS, 16, HD, 2, 6)
        api.sal_cache_resize(c, _ints([0, 1]), _ints([n, n]))
        emb[n] = api.sal_stream_prefill(x[:, :n].clone(), dw, LAYERS, c, 16, 2)
    assert rel_l2(to64(emb[40]), to64(emb[48][:, :40])) < 1e-2
    for p in range(40, 48):
        api.sal_cache_resize(caches[40], _ints([0, 1]), _ints([p + 1, p + 1]))
        e = api.sal_stream_step(x[:, p].clone(), dw, LAYERS, caches[40], 16, 2)
        assert rel_l2(to64(e), to64(emb[48][:, p])) < 1e-2
    # the caches hold the same keys and values, up to the rounding of their inputs
    for pool in ("k", "v"):
        a, b = getattr(caches[40], pool)[:, :6], getattr(caches[48], pool)[:, :6]
        assert torch.equal(caches[40].table, caches[48].table) and rel_l2(to64(a), to64(b)) < 1e-2


def test_captured_step():
    """One graph of resize and step, replayed as positions arrive; the lengths are read at replay."""
    api = _api()
    _, wf, dw = weights(LAYERS)
    S = 3
    x = torch.randn(S, 20, WIDTH, device="cuda")
    cache = api.PagedCache.empty(LAYERS, 24, HEADS, 8, HD, S, 4)
    seqs, lens, row = _ints([0, 1, 2]), _ints([0, 0, 0]), torch.zeros(S, WIDTH, device="cuda")
    emb = torch.zeros(S, WIDTH, dtype=torch.bfloat16, device="cuda")
    ws = api.stream_workspace(S)
    scratch = api.PagedCache.empty(LAYERS, 24, HEADS, 8, HD, S, 4)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # first calls outside the capture
        api.sal_cache_resize(scratch, seqs, _ints([1, 1, 1]), 10, 1)
        api.sal_stream_step(row.clone(), dw, LAYERS, scratch, 10, 1, seqs, emb, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.sal_cache_resize(cache, seqs, lens, 10, 1)
        api.sal_stream_step(row, dw, LAYERS, cache, 10, 1, seqs, emb, ws)
    for p in range(20):
        lens.fill_(p + 1)
        row.copy_(x[:, p])
        graph.replay()
        if p in (0, 7, 8, 19):
            for s in range(S):
                assert rel_l2(to64(emb[s]), _reference(x[s, :p + 1], wf, 10, 1)[-1]) < 1e-2, (p, s)
    cache.check()


def test_rows_without_a_place():
    """Sequences out of range, empty ones and a full pool: nothing is written, the others are right."""
    api = _api()
    _, wf, dw = weights(LAYERS)
    cache = api.PagedCache.empty(LAYERS, 3, HEADS, 8, HD, 3, 2)
    cache.k.zero_(), cache.v.zero_()
    x = torch.randn(4, WIDTH, device="cuda")
    api.sal_cache_resize(cache, _ints([1]), _ints([1]))
    emb = api.sal_stream_step(x.clone(), dw, LAYERS, cache, seqs=_ints([7, 1, -1, 0]))
    assert rel_l2(to64(emb[1]), _reference(x[1:2], wf, -1, 0)[-1]) < 1e-2
    used = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    used[int(cache.table[1, 0]), 0] = True
    assert not bool(cache.k.transpose(2, 3)[:, ~used].any()) and bool(cache.k.transpose(2, 3)[:, used].any())
