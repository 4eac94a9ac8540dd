"""Live-stream calls on a stream of their own while the current stream is busy, with outputs and
scratch left to the binding: both are made on the call's stream, so results neither wait for the
current stream nor are overwritten by it."""
import pytest
import torch

from gpu_util import weights

pytestmark = pytest.mark.gpu


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _forms(s):
    """The stream as an object and as a handle."""
    return (s, s.cuda_stream)


def _busy():
    torch.cuda._sleep(20_000_000)  # about 10 ms of the current stream


def _run(call, want):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for form in _forms(side):
        for _ in range(3):
            _busy()
            got = call(form)
            side.synchronize()
            torch.cuda.synchronize()
            for i, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), (i, form)
            del got


def test_windowed_attention():
    api = _api()
    q, k, v = (torch.randn(3, 10, 400, 128, device="cuda").bfloat16() for _ in range(3))
    lens = _ints([400, 0, 123])
    want = api.sal_attention_window(q, k, v, 50, 0, 2, lens)
    _run(lambda s: [api.sal_attention_window(q, k, v, 50, 0, 2, lens, stream=s)], [want])
    assert not bool(want[400:800].any())


@pytest.mark.parametrize("H,kvh", [(10, 10), (32, 2)])
def test_paged_attention(H, kvh):
    """Pieces joined inside (the workspace counts them) and by a second kernel."""
    api = _api()
    B, per = 40, 200
    k, v = (torch.randn(1, B * per, kvh, 16, 128, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(B * per, device="cuda").to(torch.int32).reshape(B, per)
    cache = api.PagedCache(k, v, table, _ints([3100 + b for b in range(B)]))
    q = torch.randn(B, H, 128, device="cuda").bfloat16()
    want = api.sal_attention_paged(q, cache)
    _run(lambda s: [api.sal_attention_paged(q, cache, stream=s)], [want])


def test_prefill_and_step():
    """(2,000 positions: the residual products of fewer rows land in no fixed order)"""
    api = _api()
    _, _, dw = weights(2)
    x = torch.randn(1, 2000, 1280, device="cuda")
    cache = api.PagedCache.empty(2, 130, 10, 16, 128, 1, 130)
    api.sal_cache_resize(cache, _ints([0]), _ints([2000]))
    want = api.sal_stream_prefill(x.clone(), dw, 2, cache, 100, 4)
    xs = [x.clone() for _ in range(6)]
    _run(lambda s: [api.sal_stream_prefill(xs.pop(), dw, 2, cache, 100, 4, stream=s)], [want])
    api.sal_cache_resize(cache, _ints([0]), _ints([2001]))
    ys = [x[:, 7].clone() for _ in range(7)]
    side = torch.cuda.Stream()
    first = api.sal_stream_step(ys.pop(), dw, 2, cache, 100, 4).double()
    torch.cuda.synchronize()
    for form in _forms(side):
        for _ in range(3):
            _busy()
            got = api.sal_stream_step(ys.pop(), dw, 2, cache, 100, 4, stream=form)
            torch.cuda.synchronize()
            assert float((got.double() - first).norm() / first.norm()) < 1e-2
    cache.check()


def test_check_waits_for_the_cache_operations():
    """An operation that fails on another stream, behind 10 ms of work there, is not missed."""
    api = _api()
    cache = api.PagedCache.empty(1, 4, 1, 8, 64, 2, 9)
    seqs, new, side = _ints([0, 1]), _ints([72, 72]), torch.cuda.Stream(priority=0)
    api.sal_cache_resize(cache, seqs, _ints([1, 1]))
    cache.check()
    with torch.cuda.stream(side):
        _busy()
    api.sal_cache_resize(cache, seqs, new, stream=side)
    with pytest.raises(RuntimeError, match="too few free pages"):
        cache.check()
    cache.check()
