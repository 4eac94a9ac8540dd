"""Thin Python binding of libsal (include/sal.h): argument marshalling over ctypes.

Every computation runs in the CUDA library; this module only allocates output buffers
with PyTorch (device memory and streams are PyTorch's), passes raw pointers, and turns
status codes into exceptions. There is no CPU fallback: if libsal.so is missing or the
device is not an sm_100 GPU, the calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsal.so")
# The bounds-checked build (sal.h, "Bounds-checked build"): same calls, every kernel's
# plain global accesses tested against the buffers it was given.
LIB_CHECKED_PATH = os.path.join(_HERE, "libsal_checked.so")

N_MELS, STACK, STACK_DIM, WIDTH, HEADS, HEAD_DIM, FFN = 128, 8, 1024, 1280, 10, 128, 5120
MAX_POSITIONS = 45000

SAL_EPI_STORE_F32, SAL_EPI_STORE_BF16, SAL_EPI_GELU_BF16, SAL_EPI_RESID_F32 = 0, 1, 2, 3

LAYER_FIELDS = ["ln1_g", "ln1_b", "w_qkv", "b_qkv", "qn_g", "kn_g", "w_o", "b_o",
                "ln2_g", "ln2_b", "w1", "b1", "w2", "b2"]


class SalError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


class sal_layer(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in LAYER_FIELDS]


class sal_weights(ctypes.Structure):
    _fields_ = [("w_proj", ctypes.c_void_p), ("b_proj", ctypes.c_void_p),
                ("layers", ctypes.POINTER(sal_layer)), ("n_layers", ctypes.c_int),
                ("lnf_g", ctypes.c_void_p), ("lnf_b", ctypes.c_void_p)]


class sal_ctc_weights(ctypes.Structure):
    _fields_ = [("w_up", ctypes.c_void_p), ("b_up", ctypes.c_void_p),
                ("layers", ctypes.POINTER(sal_layer)), ("n_layers", ctypes.c_int),
                ("lnf_g", ctypes.c_void_p), ("lnf_b", ctypes.c_void_p),
                ("w_out", ctypes.c_void_p), ("b_out", ctypes.c_void_p)]


class sal_trace(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("events", ctypes.POINTER(ctypes.c_void_p)),
                ("n_events", ctypes.c_int)]


class sal_forward_options(ctypes.Structure):
    _fields_ = [("chunk", ctypes.c_int64), ("trace", ctypes.POINTER(sal_trace)),
                ("window_core", ctypes.c_int64), ("window_context", ctypes.c_int64)]


WINDOW_CORE, WINDOW_CONTEXT = 500, 50  # the serving-window defaults (sal.h)


class sal_window(ctypes.Structure):
    _fields_ = [("left", ctypes.c_int64), ("right", ctypes.c_int64), ("sinks", ctypes.c_int64)]


class sal_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layers", ctypes.c_int), ("pages", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("sequences", ctypes.c_int), ("max_pages", ctypes.c_int), ("table", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("status", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


CACHE_NO_PAGES, CACHE_BAD_LIST, CACHE_LOST = 1, 2, 4  # bits of a cache's status word (sal.h)


KIND_NAMES = ["rope_table", "layernorm", "qkv", "attention", "out_proj", "ffn_up", "ffn_down"]

EXPORTS = {
    # name: (restype, argtypes)
    "sal_frame_count": (ctypes.c_int64, [ctypes.c_int64]),
    "sal_position_count": (ctypes.c_int64, [ctypes.c_int64]),
    "sal_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sal_frontend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p]),
    "sal_stack_project": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                          ctypes.POINTER(sal_weights), ctypes.c_void_p, ctypes.c_void_p]),
    "sal_encoder_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64]),
    "sal_encoder_workspace_bytes_ex": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64,
                                                         ctypes.POINTER(sal_forward_options)]),
    "sal_encoder_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                            ctypes.POINTER(sal_weights), ctypes.c_int, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "sal_encoder_forward_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                               ctypes.POINTER(sal_weights), ctypes.c_int, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                               ctypes.POINTER(sal_forward_options)]),
    "sal_launch_count": (ctypes.c_uint64, []),
    "sal_encode_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64]),
    "sal_encode": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(sal_weights),
                                   ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                   ctypes.c_void_p]),
    "sal_last_device_status": (ctypes.c_int, [ctypes.c_void_p]),
    "sal_weights_file_info": (ctypes.c_int, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_int),
                                              ctypes.POINTER(ctypes.c_size_t)]),
    "sal_weights_file_load": (ctypes.c_int, [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_size_t,
                                              ctypes.POINTER(sal_layer), ctypes.c_int, ctypes.POINTER(sal_weights),
                                              ctypes.c_void_p]),
    "sal_checked_build": (ctypes.c_int, []),
    "sal_check_report": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64),
                                         ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                         ctypes.POINTER(ctypes.c_uint64)]),
    "sal_check_shrink_writable": (None, [ctypes.c_uint64]),
    "sal_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "sal_layernorm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "sal_linear": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                   ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "sal_qkv_rope": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.POINTER(sal_layer),
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p]),
    "sal_qkv_rope_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                             ctypes.POINTER(sal_layer), ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p]),
    "sal_speaker_fuse": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "sal_connector": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "sal_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                      ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "sal_attention_chunked": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                              ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "sal_attention_heads": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                            ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                            ctypes.c_void_p]),
    "sal_log_softmax": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p]),
    "sal_attention_plan": (ctypes.c_int, [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "sal_attention_withhold": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                               ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                               ctypes.c_void_p]),
    "sal_ctc_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64]),
    "sal_ctc_adapter": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                        ctypes.POINTER(sal_ctc_weights), ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "sal_attention_window": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                             ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                             ctypes.POINTER(sal_window), ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p]),
    "sal_attention_window_withhold": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                                      ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                                      ctypes.POINTER(sal_window), ctypes.c_int, ctypes.c_void_p,
                                                      ctypes.c_void_p]),
    "sal_cache_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int]),
    "sal_cache_append": (ctypes.c_int, [ctypes.POINTER(sal_cache), ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p]),
    "sal_cache_copy_pages": (ctypes.c_int, [ctypes.POINTER(sal_cache), ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int, ctypes.c_void_p]),
    "sal_cache_fork": (ctypes.c_int, [ctypes.POINTER(sal_cache), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "sal_cache_resize": (ctypes.c_int, [ctypes.POINTER(sal_cache), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.POINTER(sal_window), ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p]),
    "sal_cache_compact": (ctypes.c_int, [ctypes.POINTER(sal_cache), ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p]),
    "sal_attention_paged_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(sal_cache), ctypes.c_int,
                                                               ctypes.c_int]),
    "sal_attention_paged": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                            ctypes.c_int, ctypes.POINTER(sal_cache), ctypes.c_int, ctypes.c_void_p,
                                            ctypes.POINTER(sal_window), ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_size_t, ctypes.c_void_p]),
    "sal_stream_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64]),
    "sal_stream_prefill": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                           ctypes.POINTER(sal_weights), ctypes.c_int, ctypes.POINTER(sal_window),
                                           ctypes.POINTER(sal_cache), ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "sal_stream_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(sal_weights), ctypes.c_int,
                                        ctypes.POINTER(sal_window), ctypes.POINTER(sal_cache), ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
}

_libs: dict = {}
# SAL_LIB=checked routes every call of this module through the bounds-checked build.
_active = LIB_CHECKED_PATH if os.environ.get("SAL_LIB") == "checked" else LIB_PATH


def _load(path: str) -> ctypes.CDLL:
    if path not in _libs:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: run `python -m speech_audio_encoder_b200.build`")
        l = ctypes.CDLL(path)
        for name, (res, args) in EXPORTS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _libs[path] = l
    return _libs[path]


def lib() -> ctypes.CDLL:
    """The loaded library (libsal.so, or libsal_checked.so inside `checked_library()` or
    with SAL_LIB=checked). Raises if it has not been built."""
    return _libs.get(_active) or _load(_active)


@contextlib.contextmanager
def checked_library():
    """Calls made inside this block go through libsal_checked.so."""
    global _active
    prev, _active = _active, LIB_CHECKED_PATH
    try:
        yield lib()
    finally:
        _active = prev


def status_string(status: int) -> str:
    return lib().sal_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise SalError(fn, status)


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors passed to libsal must be contiguous")
        return t.data_ptr()
    return int(t)


def _stream(stream) -> int:
    if stream is None:  # the current stream's handle, without making a Stream object for it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ----------------------------------------------------------------------------- counts

def frame_count(n_samples: int) -> int:
    return lib().sal_frame_count(int(n_samples))


def position_count(n_samples: int) -> int:
    return lib().sal_position_count(int(n_samples))


# ----------------------------------------------------------------------------- weights

class DeviceWeights:
    """Encoder parameters in one device buffer, plus the sal_weights record that points into it.

    ``w`` is the nested dict of (bf16 bits, float32) pairs from ``synth.make_weights``.
    """

    def __init__(self, w: dict, device="cuda"):
        names, arrays = [], []
        for k in ("w_proj", "b_proj", "lnf_g", "lnf_b"):
            names.append((None, k))
            arrays.append(w[k][0])
        for i, lw in enumerate(w["layers"]):
            for k in LAYER_FIELDS:
                names.append((i, k))
                arrays.append(lw[k][0])
        offsets, off = [], 0
        for a in arrays:
            offsets.append(off)
            off += (a.size + 127) // 128 * 128  # 256-byte aligned bf16 offsets
        host = np.zeros(off, dtype=np.uint16)
        for a, o in zip(arrays, offsets):
            host[o:o + a.size] = a.reshape(-1)
        self.buffer = torch.from_numpy(host.view(np.int16)).to(device).view(torch.bfloat16)
        base = self.buffer.data_ptr()
        self.n_layers = len(w["layers"])
        self._layers = (sal_layer * max(self.n_layers, 1))()
        self.ptr = {}
        for (i, k), o in zip(names, offsets):
            p = base + 2 * o
            self.ptr[(i, k)] = p
            if i is not None:
                setattr(self._layers[i], k, p)
        self.record = sal_weights(self.ptr[(None, "w_proj")], self.ptr[(None, "b_proj")],
                                  self._layers, self.n_layers, self.ptr[(None, "lnf_g")],
                                  self.ptr[(None, "lnf_b")])

    @classmethod
    def from_file(cls, path: str, device="cuda", stream=None) -> "DeviceWeights":
        """Loads a flat weight file (sal_weights_file_load) into one device buffer."""
        n_layers, nbytes = ctypes.c_int(), ctypes.c_size_t()
        _check("sal_weights_file_info", lib().sal_weights_file_info(os.fsencode(path), ctypes.byref(n_layers),
                                                                    ctypes.byref(nbytes)))
        self = cls.__new__(cls)
        self.buffer = torch.empty(nbytes.value, dtype=torch.uint8, device=device)
        self.n_layers = n_layers.value
        self._layers = (sal_layer * max(self.n_layers, 1))()
        self.record = sal_weights()
        _check("sal_weights_file_load",
               lib().sal_weights_file_load(os.fsencode(path), self.buffer.data_ptr(), nbytes.value, self._layers,
                                           self.n_layers, ctypes.byref(self.record), _stream(stream)))
        self.ptr = {(None, k): getattr(self.record, k) for k in ("w_proj", "b_proj", "lnf_g", "lnf_b")}
        for i in range(self.n_layers):
            for k in LAYER_FIELDS:
                self.ptr[(i, k)] = getattr(self._layers[i], k)
        return self

    def layer(self, i: int) -> sal_layer:
        return self._layers[i]

    def sub(self, first: int, count: int) -> sal_weights:
        """A sal_weights record over layers [first, first + count) (shares this buffer)."""
        arr = ctypes.cast(ctypes.byref(self._layers, first * ctypes.sizeof(sal_layer)),
                          ctypes.POINTER(sal_layer))
        rec = sal_weights(self.record.w_proj, self.record.b_proj, arr, count,
                          self.record.lnf_g, self.record.lnf_b)
        rec._keep = self  # keep the layer array alive
        return rec


class DeviceCtcWeights:
    """CTC adapter parameters in one device buffer, plus the sal_ctc_weights record.

    ``w`` is the dict of (bf16 bits, float32) pairs from ``synth.make_ctc_weights``; w_up
    [2, 1024, 1280] is laid out as the [2048, 1280] the library reads.
    """

    GLOBALS = ("w_up", "b_up", "lnf_g", "lnf_b", "w_out", "b_out")

    def __init__(self, w: dict, device="cuda"):
        names, arrays = [], []
        for k in self.GLOBALS:
            names.append((None, k))
            arrays.append(w[k][0])
        for i, lw in enumerate(w["layers"]):
            for k in LAYER_FIELDS:
                names.append((i, k))
                arrays.append(lw[k][0])
        offsets, off = [], 0
        for a in arrays:
            offsets.append(off)
            off += (a.size + 127) // 128 * 128
        host = np.zeros(off, dtype=np.uint16)
        for a, o in zip(arrays, offsets):
            host[o:o + a.size] = a.reshape(-1)
        self.buffer = torch.from_numpy(host.view(np.int16)).to(device).view(torch.bfloat16)
        base = self.buffer.data_ptr()
        self.n_layers = len(w["layers"])
        self._layers = (sal_layer * max(self.n_layers, 1))()
        ptr = {}
        for (i, k), o in zip(names, offsets):
            ptr[(i, k)] = base + 2 * o
            if i is not None:
                setattr(self._layers[i], k, base + 2 * o)
        g = {k: ptr[(None, k)] for k in self.GLOBALS}
        self.record = sal_ctc_weights(g["w_up"], g["b_up"], self._layers, self.n_layers, g["lnf_g"], g["lnf_b"],
                                      g["w_out"], g["b_out"])


# ----------------------------------------------------------------------------- calls

def sal_frontend(wave: torch.Tensor, stacked: bool = True, stream=None):
    """wave [batch, n] float32 (device) -> (logmel [batch, F, 128] f32, stacked [batch, T, 1024] bf16)."""
    batch, n = wave.shape
    F, T = frame_count(n), position_count(n)
    logmel = torch.empty((batch, F, N_MELS), dtype=torch.float32, device=wave.device)
    st = torch.empty((batch, T, STACK_DIM), dtype=torch.bfloat16, device=wave.device) if stacked else None
    _check("sal_frontend", lib().sal_frontend(_ptr(wave), n, batch, _ptr(logmel), _ptr(st), _stream(stream)))
    return logmel, st


def sal_stack_project(stacked: torch.Tensor, weights: DeviceWeights, stream=None) -> torch.Tensor:
    """stacked [batch, T, 1024] bf16 -> x [batch * T, 1280] float32."""
    batch, T, _ = stacked.shape
    x = torch.empty((batch * T, WIDTH), dtype=torch.float32, device=stacked.device)
    _check("sal_stack_project", lib().sal_stack_project(_ptr(stacked), batch, T, ctypes.byref(weights.record),
                                                        _ptr(x), _stream(stream)))
    return x


def encoder_workspace(batch: int, T: int, device="cuda") -> torch.Tensor:
    n = lib().sal_encoder_workspace_bytes(batch, T)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def sal_encoder_forward(x: torch.Tensor, batch: int, T: int, weights, n_layers: int,
                        workspace: torch.Tensor | None = None, emb: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """x [batch * T, 1280] f32 (clobbered: the residual stream after n_layers) -> emb bf16."""
    rec = weights.record if isinstance(weights, DeviceWeights) else weights
    if workspace is None:
        workspace = encoder_workspace(batch, T, x.device)
    if emb is None:
        emb = torch.empty((batch * T, WIDTH), dtype=torch.bfloat16, device=x.device)
    _check("sal_encoder_forward", lib().sal_encoder_forward(
        _ptr(x), batch, T, ctypes.byref(rec), n_layers, _ptr(emb), _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return emb


def encoder_workspace_ex(batch: int, T: int, chunk: int = 0, window_core: int = 0, window_context: int = 0,
                         device="cuda") -> torch.Tensor:
    opts = sal_forward_options(chunk, None, window_core, window_context)
    n = lib().sal_encoder_workspace_bytes_ex(batch, T, ctypes.byref(opts))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def sal_encoder_forward_ex(x: torch.Tensor, batch: int, T: int, weights, n_layers: int,
                           workspace: torch.Tensor | None = None, emb: torch.Tensor | None = None,
                           chunk: int = 0, kind: int | None = None, events=None, stream=None,
                           window_core: int = 0, window_context: int = 0) -> torch.Tensor:
    """sal_encoder_forward with chunked attention (``chunk`` positions per chunk, 0 = whole
    clip) or serving windows (``window_core`` core positions with ``window_context`` context
    positions on each side, 0 = none) and, optionally, torch.cuda.Event pairs recorded
    around each launch of ``kind``."""
    rec = weights.record if isinstance(weights, DeviceWeights) else weights
    if workspace is None:
        workspace = encoder_workspace_ex(batch, T, chunk, window_core, window_context, x.device)
    if emb is None:
        emb = torch.empty((batch * T, WIDTH), dtype=torch.bfloat16, device=x.device)
    trace_p = None
    if events:
        if any(e.cuda_event == 0 for e in events):
            raise ValueError("record each torch.cuda.Event once before tracing (its handle is created lazily)")
        handles = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
        tr = sal_trace(kind, ctypes.cast(handles, ctypes.POINTER(ctypes.c_void_p)), len(events))
        trace_p = ctypes.pointer(tr)
    opts = sal_forward_options(chunk, trace_p, window_core, window_context)
    _check("sal_encoder_forward_ex", lib().sal_encoder_forward_ex(
        _ptr(x), batch, T, ctypes.byref(rec), n_layers, _ptr(emb), _ptr(workspace), workspace.numel(),
        _stream(stream), ctypes.byref(opts)))
    return emb


def sal_launch_count() -> int:
    return int(lib().sal_launch_count())


def encode_workspace(batch: int, n_samples: int, device="cuda") -> torch.Tensor:
    n = lib().sal_encode_workspace_bytes(batch, n_samples)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def sal_encode(wave: torch.Tensor, weights: DeviceWeights, n_layers: int, emb: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Whole path; ``wave`` and ``emb`` may live on the host (pinned or not) or the device."""
    batch, n = wave.shape
    T = position_count(n)
    if workspace is None:
        workspace = encode_workspace(batch, n)
    if emb is None:
        emb = torch.empty((batch, T, WIDTH), dtype=torch.bfloat16, device=wave.device)
    _check("sal_encode", lib().sal_encode(_ptr(wave), n, batch, ctypes.byref(weights.record), n_layers,
                                          _ptr(emb), _ptr(workspace), workspace.numel(), _stream(stream)))
    return emb


def sal_layernorm(x: torch.Tensor, g: int, b: int, stream=None) -> torch.Tensor:
    y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _check("sal_layernorm", lib().sal_layernorm(_ptr(x), x.shape[0], g, b, _ptr(y), _stream(stream)))
    return y


def sal_linear(epilogue: int, A: torch.Tensor, W: torch.Tensor, bias: torch.Tensor,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M, K = A.shape
    N = W.shape[0]
    if out is None:
        dt = torch.float32 if epilogue in (SAL_EPI_STORE_F32, SAL_EPI_RESID_F32) else torch.bfloat16
        out = torch.empty((M, N), dtype=dt, device=A.device)
    _check("sal_linear", lib().sal_linear(epilogue, _ptr(A), M, K, _ptr(W), N, _ptr(bias), _ptr(out),
                                          _stream(stream)))
    return out


def sal_qkv_rope(h: torch.Tensor, batch: int, T: int, layer: sal_layer, stream=None):
    shape = (batch, HEADS, T, HEAD_DIM)
    q = torch.empty(shape, dtype=torch.bfloat16, device=h.device)
    k = torch.empty_like(q)
    v = torch.empty_like(q)
    cs = torch.empty((2, T, 64), dtype=torch.float32, device=h.device)
    _check("sal_qkv_rope", lib().sal_qkv_rope(_ptr(h), batch, T, ctypes.byref(layer), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(cs), _stream(stream)))
    return q, k, v


def sal_qkv_rope_noalloc(h: torch.Tensor, batch: int, T: int, layer: sal_layer, q: torch.Tensor,
                         k: torch.Tensor, v: torch.Tensor, stream=None):
    """sal_qkv_rope into caller-provided q, k, v [batch, 10, T, 128] bf16; allocates nothing."""
    _check("sal_qkv_rope_noalloc", lib().sal_qkv_rope_noalloc(_ptr(h), batch, T, ctypes.byref(layer), _ptr(q),
                                                              _ptr(k), _ptr(v), _stream(stream)))
    return q, k, v


def sal_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None) -> torch.Tensor:
    batch, H, T, hd = q.shape
    o = torch.empty((batch * T, H * hd), dtype=torch.bfloat16, device=q.device)
    _check("sal_attention", lib().sal_attention(_ptr(q), _ptr(k), _ptr(v), batch, T, _ptr(o), _stream(stream)))
    return o


def sal_attention_withhold(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kernel: int, tile: int,
                           stream=None) -> torch.Tensor:
    """Test hook: sal_attention with key/value tile ``tile`` of every CTA never loaded, so a
    bounded wait gives up (read the outcome with sal_last_device_status)."""
    batch, H, T, hd = q.shape
    o = torch.empty((batch * T, H * hd), dtype=torch.bfloat16, device=q.device)
    _check("sal_attention_withhold", lib().sal_attention_withhold(_ptr(q), _ptr(k), _ptr(v), batch, T, kernel, tile,
                                                                  _ptr(o), _stream(stream)))
    return o


def sal_attention_chunked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, chunk: int, stream=None) -> torch.Tensor:
    batch, H, T, hd = q.shape
    o = torch.empty((batch * T, H * hd), dtype=torch.bfloat16, device=q.device)
    _check("sal_attention_chunked", lib().sal_attention_chunked(_ptr(q), _ptr(k), _ptr(v), batch, T, chunk,
                                                                _ptr(o), _stream(stream)))
    return o


def sal_speaker_fuse(H: torch.Tensor, P: torch.Tensor, g: torch.Tensor, b: torch.Tensor,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """H [rows, 1280] bf16, P [rows, 8] f32 -> H + LN_8(P > 0.5) K (bf16)."""
    if out is None:
        out = torch.empty_like(H)
    _check("sal_speaker_fuse", lib().sal_speaker_fuse(_ptr(H), _ptr(P), H.shape[0], _ptr(g), _ptr(b), _ptr(out),
                                                      _stream(stream)))
    return out


def sal_connector(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor, stream=None) -> torch.Tensor:
    """x [rows, 1280] bf16 -> [rows, 2688] bf16."""
    out = torch.empty((x.shape[0], 2688), dtype=torch.bfloat16, device=x.device)
    _check("sal_connector", lib().sal_connector(_ptr(x), x.shape[0], _ptr(W), _ptr(bias), _ptr(out),
                                                _stream(stream)))
    return out


def sal_last_device_status(stream=None) -> int:
    return lib().sal_last_device_status(_stream(stream))


def sal_set_wait_limit_ns(ns: int) -> None:
    lib().sal_set_wait_limit_ns(int(ns))


FILE_IDS = {1: "frontend.cu", 2: "rowops.cu", 3: "gemm.cu", 4: "attention.cu", 5: "ctc.cu",
            6: "window_attention.cu", 7: "paged_attention.cu", 8: "cache.cu", 9: "stream.cu"}


def check_report() -> dict:
    """Reads and clears the checked build's record of refused accesses (sal_check_report)."""
    count, addr, seq = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
    f, ln = ctypes.c_int(), ctypes.c_int()
    _check("sal_check_report", lib().sal_check_report(ctypes.byref(count), ctypes.byref(addr), ctypes.byref(f),
                                                       ctypes.byref(ln), ctypes.byref(seq)))
    return {"count": count.value, "first_address": addr.value, "file": FILE_IDS.get(f.value, f.value),
            "line": ln.value, "first_launch": seq.value}


def check_shrink_writable(nbytes: int) -> None:
    """Test hook of the checked build: writable ranges declared from now on end nbytes early."""
    lib().sal_check_shrink_writable(int(nbytes))


CTC_CLASSES = 23863


def ctc_workspace(batch: int, T: int, device="cuda") -> torch.Tensor:
    n = lib().sal_ctc_workspace_bytes(batch, T)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def sal_ctc_adapter(h: torch.Tensor, batch: int, T: int, weights: DeviceCtcWeights,
                    logp: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Unfused encoder states h [batch * T, 1280] bf16 -> log-probabilities
    [batch * 2T, 23863] float32 on the 40 ms grid."""
    if logp is None:
        logp = torch.empty((batch * 2 * T, CTC_CLASSES), dtype=torch.float32, device=h.device)
    if workspace is None:
        workspace = ctc_workspace(batch, T, h.device)
    _check("sal_ctc_adapter", lib().sal_ctc_adapter(_ptr(h), batch, T, ctypes.byref(weights.record), _ptr(logp),
                                                    _ptr(workspace), workspace.numel(), _stream(stream)))
    return logp


def sal_attention_heads(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None) -> torch.Tensor:
    """q, k, v [batch, heads, T, head_dim] bf16 (head_dim 64 or 128) -> o [batch, T, heads * head_dim]."""
    B, H, T, hd = q.shape
    o = torch.empty((B, T, H * hd), dtype=torch.bfloat16, device=q.device)
    _check("sal_attention_heads", lib().sal_attention_heads(_ptr(q), _ptr(k), _ptr(v), B, T, H, hd, _ptr(o),
                                                            _stream(stream)))
    return o


def sal_log_softmax(z: torch.Tensor, n: int | None = None, stream=None) -> torch.Tensor:
    """Row log-softmax of the first n columns of z [rows, ld] float32 -> [rows, n]."""
    rows, ld = z.shape
    n = ld if n is None else n
    out = torch.empty((rows, n), dtype=torch.float32, device=z.device)
    _check("sal_log_softmax", lib().sal_log_softmax(_ptr(z), rows, n, ld, _ptr(out), _stream(stream)))
    return out


def attention_plan(batch: int, T: int, heads: int = 10, head_dim: int = 128, sms: int = 148) -> tuple[int, int]:
    """(pairs for the two-tile kernel, query tiles per clip) that sal_attention would use."""
    p, q = ctypes.c_int(), ctypes.c_int()
    _check("sal_attention_plan", lib().sal_attention_plan(batch, T, heads, head_dim, sms, ctypes.byref(p),
                                                          ctypes.byref(q)))
    return p.value, q.value


# ----------------------------------------------------------------------------- live streams

_windows: dict = {}


def _no_device() -> int:
    raise RuntimeError("this torch was built without CUDA")


_current_device = getattr(torch._C, "_cuda_getDevice", _no_device)  # (host-side calls need none)


def _window(left: int, right: int, sinks: int):
    """The sal_window of these limits, by reference (made once: a step of a stream asks for the same one every time)."""
    w = _windows.get((left, right, sinks))
    if w is None:
        if len(_windows) > 1000:
            _windows.clear()
        w = _windows[(left, right, sinks)] = ctypes.byref(sal_window(left, right, sinks))
    return w


def _operand(name: str, t: torch.Tensor, dtype, shape=None) -> int:
    """The address of a contiguous tensor of this type (and shape) on the current device."""
    if t.dtype is not dtype or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: expected {dtype}{'' if shape is None else ' of shape ' + str(tuple(shape))}, got "
                         f"{t.dtype} of shape {tuple(t.shape)}")
    if t.get_device() != _current_device():
        raise ValueError(f"{name}: must be on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libsal must be contiguous")
    return t.data_ptr()


def _list_operand(name: str, t: torch.Tensor | None, n: int | None = None) -> int:
    """The address of a one-dimensional int32 device tensor (of n entries), 0 for None."""
    if t is None:
        return 0
    if t.dim() != 1:
        raise ValueError(f"{name}: expected one dimension, got {t.dim()}")
    return _operand(name, t, torch.int32, None if n is None else (n,))


def _made(make, stream, returned: bool):
    """make(): a tensor that the caller of a call on `stream` did not bring, allocated and filled on that stream, so
    that the call's kernels come behind its fill and whatever gets its memory next comes behind them. One that is
    returned is used on the current stream too: its memory then waits for both."""
    if stream is None:
        return make()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) > 1 else torch.cuda.default_stream()
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = make()
    if returned and t.is_cuda:
        t.record_stream(current)
    return t


def sal_attention_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, left: int = -1, right: int = -1,
                         sinks: int = 0, lengths: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """q [batch, heads, T, head_dim], k and v [batch, kv_heads, T, head_dim] bf16 -> o [batch * T, heads * head_dim]:
    position p sees the keys j <= p + right with j >= p - left or j < sinks (a negative left or right is no limit).
    ``lengths`` [batch] int32: positions of each clip; rows of ``out`` past them are left as they were (a tensor made
    here starts as zeros then)."""
    B, H, T, hd = q.shape
    kvh = k.shape[1] if k.dim() == 4 else 0
    if out is None:
        out = _made(lambda: (torch.empty if lengths is None else torch.zeros)((B * T, H * hd), dtype=torch.bfloat16,
                                                                              device=q.device), stream, True)
    kv = (B, kvh, T, hd)
    _check("sal_attention_window", lib().sal_attention_window(
        _operand("q", q, torch.bfloat16), _operand("k", k, torch.bfloat16, kv), _operand("v", v, torch.bfloat16, kv), B,
        T, H, kvh, hd, _window(left, right, sinks), _list_operand("lengths", lengths, B),
        _operand("out", out, torch.bfloat16, (B * T, H * hd)), _stream(stream)))
    return out


def sal_attention_window_withhold(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, tile: int, left: int = -1,
                                  right: int = -1, sinks: int = 0, stream=None) -> torch.Tensor:
    """Test hook: sal_attention_window with no key tile from ``tile`` on ever loaded, so a bounded wait gives up (read
    the outcome with sal_last_device_status)."""
    B, H, T, hd = q.shape
    o = _made(lambda: torch.empty((B * T, H * hd), dtype=torch.bfloat16, device=q.device), stream, True)
    _check("sal_attention_window_withhold", lib().sal_attention_window_withhold(
        _operand("q", q, torch.bfloat16), _operand("k", k, torch.bfloat16, q.shape),
        _operand("v", v, torch.bfloat16, q.shape), B, T, H, hd, _window(left, right, sinks), tile, o.data_ptr(), _stream(stream)))
    return o


class PagedCache:
    """Keys and values of live sequences in pages (sal_cache in sal.h), in the caller's tensors:

    k, v [layers, pages, kv_heads, page_size, head_dim] bf16, table [sequences, max_pages] int32 and lengths
    [sequences] int32 (the tables are the whole state: a page that no row uses is free). ``empty`` makes a cache
    without sequences; ``with_tables`` makes another view of the same pages, for calls that leave the old tables valid.
    Failed operations set bits of ``status`` (CACHE_NO_PAGES, CACHE_BAD_LIST, CACHE_LOST); ``check`` reads it.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                 status: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
        layers, pages, kv_heads, page_size, head_dim = k.shape
        sequences, max_pages = table.shape
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=k.device)
        if workspace is None:
            n = lib().sal_cache_workspace_bytes(pages, sequences)
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=k.device)
        self.k, self.v, self.table, self.lengths = k, v, table, lengths
        self.status, self.workspace = status, workspace
        self.kv_heads, self.head_dim = kv_heads, head_dim
        self.record = sal_cache(
            _operand("k", k, torch.bfloat16), _operand("v", v, torch.bfloat16, k.shape), layers, pages, kv_heads,
            page_size, head_dim, sequences, max_pages, _operand("table", table, torch.int32),
            _operand("lengths", lengths, torch.int32, (sequences,)), _operand("status", status, torch.int32, (1,)),
            _operand("workspace", workspace, torch.uint8), workspace.numel())
        self.device_index, self._ref = k.get_device(), ctypes.byref(self.record)
        self.pool, self.places = k.data_ptr(), (self.record.table, self.record.lengths)

    @property
    def ref(self):
        """The record by reference, for a call on the current device."""
        if self.device_index != _current_device():
            raise ValueError("cache: must be on the current CUDA device")
        return self._ref

    @classmethod
    def empty(cls, layers: int, pages: int, kv_heads: int, page_size: int, head_dim: int, sequences: int,
              max_pages: int, device="cuda") -> "PagedCache":
        shape = (layers, pages, kv_heads, page_size, head_dim)
        return cls(torch.empty(shape, dtype=torch.bfloat16, device=device),
                   torch.empty(shape, dtype=torch.bfloat16, device=device),
                   torch.full((sequences, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(sequences, dtype=torch.int32, device=device))

    def with_tables(self, table: torch.Tensor, lengths: torch.Tensor) -> "PagedCache":
        """The same pages under other tables of the same shape."""
        if table.shape != self.table.shape:
            raise ValueError("with_tables: the tables must have the cache's shape")
        return PagedCache(self.k, self.v, table, lengths, self.status, self.workspace)

    def check(self) -> None:
        """Waits for the device and raises if an operation has failed since the last check."""
        torch.cuda.synchronize(self.status.device)  # the operations may run on other streams than the current one
        bits = int(self.status.item())
        if bits:
            self.status.zero_()
            torch.cuda.synchronize(self.status.device)
            what = [w for b, w in ((CACHE_NO_PAGES, "too few free pages"),
                                   (CACHE_BAD_LIST, "a list with an index or length out of range, or a sequence twice"),
                                   (CACHE_LOST, "growth from inside a page that has been let go"))
                    if bits & b]
            raise RuntimeError("cache operation failed: " + "; ".join(what))

    def _tables_of(self, out: "PagedCache | None") -> tuple:
        if out is None:
            return self, *self.places
        if out.table.shape != self.table.shape or out.pool != self.pool:
            raise ValueError("out: must be this cache's pages under tables of the same shape")
        return out, *out.places


def sal_cache_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor | None,
                     seqs: torch.Tensor | None = None, layer: int = 0, stream=None) -> None:
    """k, v [batch, kv_heads, T, head_dim] bf16 into positions starts[b] + t (None: t) of sequences seqs[b] (None: b).
    Two tokens for one position leave unspecified contents there."""
    B, kvh, T, hd = k.shape
    if kvh != cache.kv_heads or hd != cache.head_dim:
        raise ValueError(f"k: the cache has {cache.kv_heads} heads of {cache.head_dim}")
    _check("sal_cache_append", lib().sal_cache_append(
        cache.ref, layer, _operand("k", k, torch.bfloat16), _operand("v", v, torch.bfloat16, k.shape), B, T,
        _list_operand("starts", starts, B), _list_operand("seqs", seqs, B), _stream(stream)))


def sal_cache_copy_pages(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Page src[i] to page dst[i] in every layer (the tables are not touched)."""
    n = src.shape[0]
    _check("sal_cache_copy_pages", lib().sal_cache_copy_pages(
        cache.ref, _list_operand("src", src), _list_operand("dst", dst, n), n, _stream(stream)))


def sal_cache_fork(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor, out: PagedCache | None = None,
                   stream=None) -> PagedCache:
    """Sequences dst[i] become forks of src[i]; the new tables go to ``out`` (None: in place)."""
    out, table, lengths = cache._tables_of(out)
    n = src.shape[0]
    _check("sal_cache_fork", lib().sal_cache_fork(
        cache.ref, _list_operand("src", src), _list_operand("dst", dst, n), n, table, lengths, _stream(stream)))
    return out


def sal_cache_resize(cache: PagedCache, seqs: torch.Tensor, new_lengths: torch.Tensor, left: int = -1, sinks: int = 0,
                     out: PagedCache | None = None, stream=None) -> PagedCache:
    """Sequences seqs[i] get the length new_lengths[i] (0 frees them); with left >= 0 the pages that no later
    position sees are let go. The new tables go to ``out`` (None: in place)."""
    out, table, lengths = cache._tables_of(out)
    n = seqs.shape[0]
    _check("sal_cache_resize", lib().sal_cache_resize(
        cache.ref, _list_operand("seqs", seqs), _list_operand("new_lengths", new_lengths, n), n, _window(left, 0, sinks),
        table, lengths, _stream(stream)))
    return out


def sal_cache_compact(cache: PagedCache, out: PagedCache | None = None, stream=None) -> PagedCache:
    """Moves the pages in use to the lowest numbers; the new tables go to ``out`` (None: in place)."""
    out, table, lengths = cache._tables_of(out)
    _check("sal_cache_compact", lib().sal_cache_compact(cache.ref, table, lengths, _stream(stream)))
    return out


def attention_paged_workspace(cache: PagedCache, batch: int, heads: int) -> torch.Tensor:
    """Scratch of sal_attention_paged (zero-filled on the current stream, as its first use needs it)."""
    n = lib().sal_attention_paged_workspace_bytes(cache._ref, batch, heads)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=cache.k.device)


def sal_attention_paged(q: torch.Tensor, cache: PagedCache, left: int = -1, sinks: int = 0, layer: int = 0,
                        seqs: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [batch, heads, head_dim] bf16 (any strides of its first two dimensions that are multiples of 8), the newest
    position of sequences seqs[b] (None: b) -> o [batch, heads * head_dim]."""
    B, H, hd = q.shape
    rows, heads, inner = q.stride()
    if hd != cache.head_dim or inner != 1:
        raise ValueError(f"q: expected contiguous heads of {cache.head_dim}")
    if q.dtype is not torch.bfloat16 or q.get_device() != _current_device():
        raise ValueError("q: expected bfloat16 on the current CUDA device")
    if out is None:
        out = _made(lambda: torch.empty((B, H * hd), dtype=torch.bfloat16, device=q.device), stream, True)
    if workspace is None:
        workspace = _made(lambda: attention_paged_workspace(cache, B, H), stream, False)
    _check("sal_attention_paged", lib().sal_attention_paged(
        q.data_ptr(), rows, heads, B, H, cache.ref, layer, 0 if seqs is None else _list_operand("seqs", seqs, B),
        _window(left, 0, sinks), _operand("out", out, torch.bfloat16, (B, H * hd)),
        _operand("workspace", workspace, torch.uint8), workspace.numel(), _stream(stream)))
    return out


def stream_workspace(batch: int, T: int = 1, device="cuda") -> torch.Tensor:
    """Scratch of sal_stream_prefill over T positions (1: of sal_stream_step)."""
    n = lib().sal_stream_workspace_bytes(batch, T)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def sal_stream_prefill(x: torch.Tensor, weights, n_layers: int, cache: PagedCache, left: int = -1, sinks: int = 0,
                       lengths: torch.Tensor | None = None, seqs: torch.Tensor | None = None,
                       emb: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """x [batch, T, 1280] float32 (clobbered): the first positions of live streams -> emb [batch, T, 1280] bf16, their
    keys and values kept in the cache (resize the sequences first; nothing is kept while ``cache.status`` is set)."""
    rec = weights.record if isinstance(weights, DeviceWeights) else weights
    B, T, width = x.shape
    if emb is None:
        emb = _made(lambda: torch.empty((B, T, width), dtype=torch.bfloat16, device=x.device), stream, True)
    if workspace is None:
        workspace = _made(lambda: stream_workspace(B, T, x.device), stream, False)
    _check("sal_stream_prefill", lib().sal_stream_prefill(
        _operand("x", x, torch.float32, (B, T, WIDTH)), B, T, _list_operand("lengths", lengths, B), ctypes.byref(rec),
        n_layers, _window(left, 0, sinks), cache.ref, _list_operand("seqs", seqs, B),
        _operand("emb", emb, torch.bfloat16, x.shape), _operand("workspace", workspace, torch.uint8),
        workspace.numel(), _stream(stream)))
    return emb


def sal_stream_step(x: torch.Tensor, weights, n_layers: int, cache: PagedCache, left: int = -1, sinks: int = 0,
                    seqs: torch.Tensor | None = None, emb: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x [batch, 1280] float32 (clobbered): one new position of each live stream -> emb [batch, 1280] bf16 (make the
    sequences longer by one first, with sal_cache_resize; nothing is kept while ``cache.status`` is set, as a resize
    that failed does)."""
    rec = weights.record if isinstance(weights, DeviceWeights) else weights
    B, width = x.shape
    if emb is None:
        emb = _made(lambda: torch.empty((B, width), dtype=torch.bfloat16, device=x.device), stream, True)
    if workspace is None:
        workspace = _made(lambda: stream_workspace(B, 1, x.device), stream, False)
    _check("sal_stream_step", lib().sal_stream_step(
        _operand("x", x, torch.float32, (B, WIDTH)), B, ctypes.byref(rec), n_layers, _window(left, 0, sinks), cache.ref,
        _list_operand("seqs", seqs, B), _operand("emb", emb, torch.bfloat16, x.shape),
        _operand("workspace", workspace, torch.uint8), workspace.numel(), _stream(stream)))
    return emb
