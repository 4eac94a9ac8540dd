"""The binding of the live-stream calls on the CPU, with a library that only records what it is
given: on which stream the tensors are made that a caller leaves out."""
import contextlib
import os
import subprocess
import sys

import pytest
import torch

from speech_audio_encoder_b200 import api


class FakeLib:
    """Every call succeeds; sizes are 4096 bytes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_bytes") else 0
        return call


class FakeStream:
    cuda_stream = 0x7000


@pytest.fixture
def fake(monkeypatch):
    """CPU tensors pass for ones on the current device (-1). Records (maker, stream it was made on)."""
    lib, now, made = FakeLib(), [None], []
    monkeypatch.setattr(api, "lib", lambda: lib)
    monkeypatch.setattr(api, "_current_device", lambda: -1)
    monkeypatch.setattr(api, "_stream", lambda s: 0 if s is None else s.cuda_stream)

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    for name in ("empty", "zeros", "full"):
        def maker(*a, _make=getattr(torch, name), _name=name, **kw):
            made.append((_name, now[-1]))
            return _make(*a, **kw)
        monkeypatch.setattr(torch, name, maker)
    lib.made = made
    return lib


def _bf16(*shape):
    return torch.ones(shape, dtype=torch.bfloat16)


def _ints(n):
    return torch.ones(n, dtype=torch.int32)


def _cache(layers=1):
    return api.PagedCache(_bf16(layers, 2, 10, 8, 128), _bf16(layers, 2, 10, 8, 128), torch.ones(2, 3, dtype=torch.int32),
                          _ints(2))


def _calls(stream):
    """Each live-stream call that makes tensors of its own, with everything left out."""
    q, x, rec = _bf16(2, 10, 5, 128), torch.ones(2, 5, 1280), api.sal_weights()
    cache = _cache()
    return {
        "window": lambda: api.sal_attention_window(q, q, q, stream=stream),
        "window with lengths": lambda: api.sal_attention_window(q, q, q, lengths=_ints(2), stream=stream),
        "withhold": lambda: api.sal_attention_window_withhold(q, q, q, 1, stream=stream),
        "paged": lambda: api.sal_attention_paged(_bf16(2, 10, 128), cache, stream=stream),
        "prefill": lambda: api.sal_stream_prefill(x, rec, 0, cache, stream=stream),
        "step": lambda: api.sal_stream_step(torch.ones(2, 1280), rec, 0, cache, stream=stream),
    }


NAMES = ["window", "window with lengths", "withhold", "paged", "prefill", "step"]


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_makes_belongs_to_its_stream(fake, name):
    """A fill on the current stream could land behind the kernel that runs on the other, and memory
    that goes back to the current stream could be handed out while that kernel still uses it."""
    for stream in (FakeStream(), None):
        call = _calls(stream)[name]
        fake.made.clear()
        call()
        assert fake.made and all(on is stream for _, on in fake.made), fake.made
        assert fake.calls[-1][1][-1] == (0 if stream is None else stream.cuda_stream)


def test_the_binding_imports_where_torch_has_no_cuda():
    """Host-side calls work on a torch that was built without CUDA functions."""
    code = ("import torch\n"
            "for name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    delattr(torch._C, name)\n"
            "from speech_audio_encoder_b200 import api, build\n"
            "build.build(quiet=True)\n"
            "assert api.sal_cache and api.position_count(16000) > 0\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True)


def test_a_cache_on_another_device_is_refused(fake, monkeypatch):
    """Its addresses mean nothing to the current device: no call is made with them."""
    cache, q, x, rec = _cache(), _bf16(2, 10, 128), torch.ones(2, 1280), api.sal_weights()
    kv = _bf16(1, 10, 1, 128)
    on_two = torch.empty(1, dtype=torch.int8)  # stands for an operand on the current device, 2

    class Other(torch.Tensor):
        def get_device(self):
            return 2

    def there(t):
        return t.as_subclass(Other)

    monkeypatch.setattr(api, "_current_device", lambda: 2)
    assert there(on_two).get_device() == 2
    fake.calls.clear()
    lists = there(_ints(1))
    for call in (lambda: api.sal_cache_compact(cache), lambda: api.sal_cache_fork(cache, lists, lists),
                 lambda: api.sal_cache_resize(cache, lists, lists), lambda: api.sal_cache_copy_pages(cache, lists, lists),
                 lambda: api.sal_cache_append(cache, there(kv), there(kv), None),
                 lambda: api.sal_attention_paged(there(q), cache, out=there(_bf16(2, 1280)),
                                                 workspace=there(torch.ones(4096, dtype=torch.uint8))),
                 lambda: api.sal_stream_prefill(there(x[:, None].contiguous()), rec, 0, cache, emb=there(_bf16(2, 1, 1280)),
                                                workspace=there(torch.ones(4096, dtype=torch.uint8))),
                 lambda: api.sal_stream_step(there(x), rec, 0, cache, emb=there(_bf16(2, 1280)),
                                             workspace=there(torch.ones(4096, dtype=torch.uint8)))):
        with pytest.raises(ValueError, match="device"):
            call()
    assert not fake.calls
