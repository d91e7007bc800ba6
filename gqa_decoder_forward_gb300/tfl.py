"""Thin Python binding of libtfl.so (include/tfl.h).

Argument marshalling only: every step of the forward runs in the library's CUDA
kernels.  PyTorch supplies device memory (tensors whose data_ptr is passed through)
and streams.  Functions keep the C names; the small classes below only own the
tensors that back a model's workspace and KV buffers.

The library is required: importing this module without a built libtfl.so raises,
and nothing here falls back to another implementation.
"""
from __future__ import annotations

import ctypes
import operator
import os
from typing import Sequence

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtfl.so")

TFL_OK = 0
TFL_E_GEOMETRY = -1
TFL_E_ARCH = -2
TFL_E_CAPACITY = -3
TFL_E_ARG = -4
TFL_E_CUDA = -5
TFL_E_NONFINITE = -6
TFL_E_WORKSPACE = -7
TFL_E_DEVICE = -8
TFL_KV_PAGE = 128

_vp = ctypes.c_void_p
_intp = ctypes.POINTER(ctypes.c_int)


class tfl_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("layers", ctypes.c_int), ("n_q", ctypes.c_int),
                ("n_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("vocab", ctypes.c_int), ("rope_theta", ctypes.c_double), ("rms_eps", ctypes.c_float),
                ("max_rows", ctypes.c_int), ("max_decode_rows", ctypes.c_int), ("max_context", ctypes.c_int)]


class tfl_draft_stats(ctypes.Structure):
    _fields_ = [("rounds", ctypes.c_longlong), ("drafted", ctypes.c_longlong), ("accepted", ctypes.c_longlong),
                ("target_rows", ctypes.c_longlong), ("drafter_rows", ctypes.c_longlong)]


class tfl_weights(ctypes.Structure):
    _fields_ = [("embed", _vp), ("final_norm", _vp), ("lm_head", _vp)] + [
        (n, ctypes.POINTER(_vp)) for n in
        ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "wg", "wu", "wd")]


# C symbol -> (restype, argtypes); every symbol include/tfl.h declares
SIGNATURES = {
    "tfl_qualify": (ctypes.c_int, [ctypes.POINTER(tfl_config), ctypes.c_char_p, ctypes.c_size_t]),
    "tfl_rope_table": (None, [ctypes.c_double, ctypes.c_int, _vp, _vp]),
    "tfl_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(tfl_config)]),
    "tfl_init": (ctypes.c_int, [ctypes.POINTER(tfl_config), ctypes.POINTER(tfl_weights), _vp, ctypes.c_size_t,
                                ctypes.POINTER(_vp)]),
    "tfl_free": (None, [_vp]),
    "tfl_last_error": (ctypes.c_char_p, []),
    "tfl_error_string": (ctypes.c_char_p, [ctypes.c_int]),
    "tfl_kv_bytes": (ctypes.c_size_t, [ctypes.POINTER(tfl_config), ctypes.c_int]),
    "tfl_kv_alloc": (ctypes.c_int, [_vp, ctypes.c_int, _vp, ctypes.c_size_t, ctypes.POINTER(_vp)]),
    "tfl_kv_free": (None, [_vp]),
    "tfl_kv_reset": (ctypes.c_int, [_vp, ctypes.c_int]),
    "tfl_kv_length": (ctypes.c_int, [_vp]),
    "tfl_kv_capacity": (ctypes.c_int, [_vp]),
    "tfl_kv_write": (ctypes.c_int, [_vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]),
    "tfl_kv_read": (ctypes.c_int, [_vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]),
    "tfl_decode_step": (ctypes.c_int, [_vp, ctypes.POINTER(_vp), ctypes.c_int, _vp, ctypes.POINTER(ctypes.c_int),
                                       _vp, _vp]),
    "tfl_prefill_chunk": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp]),
    "tfl_argmax": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp]),
    "tfl_status": (ctypes.c_int, [_vp, _vp]),
    "tfl_wait_probe": (ctypes.c_int, [_vp, ctypes.c_int, ctypes.c_int, _vp]),
    "tfl_decode_hidden": (ctypes.c_int, [_vp, ctypes.POINTER(_vp), ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                         _vp, _vp, _vp]),
    "tfl_prefill_hidden": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _vp, _vp]),
    "tfl_head": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp]),
    "tfl_layer_op": (ctypes.c_int, [_vp, ctypes.c_int, ctypes.c_int, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp,
                                    _vp]),
    "tfl_attention_decode_noalloc": (ctypes.c_int, [_vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]),
    "tfl_profile": (ctypes.c_int, [_vp, ctypes.c_int]),
    "tfl_set_persistent": (ctypes.c_int, [_vp, ctypes.c_int]),
    "tfl_kv_copy_prefix": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _vp]),
    "tfl_prefix_store_new": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(_vp)]),
    "tfl_prefix_store_free": (None, [_vp]),
    "tfl_prefix_store_put": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_int32), ctypes.c_int, _vp]),
    "tfl_prefix_store_match": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_int32), ctypes.c_int,
                                              ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_int)]),
    "tfl_prefix_store_remove": (ctypes.c_int, [_vp, _vp]),
    "tfl_prefix_store_size": (ctypes.c_int, [_vp]),
    "tfl_sample": (ctypes.c_int, [_vp, _vp, ctypes.c_int, ctypes.c_float, ctypes.c_int, ctypes.c_float, _vp, _vp,
                                  _vp]),
    "tfl_step_phases": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_double), ctypes.c_int]),
    "tfl_drafted_workspace_bytes": (ctypes.c_size_t, [_vp, ctypes.c_int]),
    "tfl_decode_drafted": (ctypes.c_int, [_vp, _vp, _vp, _vp, ctypes.c_int, ctypes.POINTER(ctypes.c_int32),
                                          ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int32), _vp,
                                          ctypes.c_size_t, _vp, _vp]),
    "tfl_copy_draft": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_int,
                                      ctypes.POINTER(ctypes.c_int32)]),
    "tfl_profile_read": (ctypes.c_int, [_vp, ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_long)]),
    "tfl_profile_kind": (ctypes.c_char_p, [ctypes.c_int]),
    "tfl_kv4_bytes": (ctypes.c_size_t, [ctypes.c_int] * 4),
    "tfl_kv4_alloc": (ctypes.c_int, [ctypes.c_int] * 4 + [_vp, ctypes.c_size_t, ctypes.POINTER(_vp)]),
    "tfl_kv4_free": (None, [_vp]),
    "tfl_kv4_reset": (ctypes.c_int, [_vp, ctypes.c_int]),
    "tfl_kv4_length": (ctypes.c_int, [_vp]),
    "tfl_kv4_capacity": (ctypes.c_int, [_vp]),
    # arrays as addresses, which cost less per call than typed pointers (see KV4Rows)
    "tfl_kv4_write": (ctypes.c_int, [_vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp,
                                     ctypes.c_size_t, _vp]),
    "tfl_kv4_read": (ctypes.c_int, [_vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp,
                                    ctypes.c_size_t, _vp]),
    "tfl_kv4_attn_bytes": (ctypes.c_size_t, [ctypes.c_int] * 5),
    "tfl_kv4_attn_init": (ctypes.c_int, [ctypes.c_int] * 5 + [_vp, ctypes.c_size_t, ctypes.POINTER(_vp)]),
    "tfl_kv4_attn_free": (None, [_vp]),
    "tfl_kv4_attn_status": (ctypes.c_int, [_vp, _vp]),
    "tfl_kv4_attention": (ctypes.c_int, [_vp, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp,
                                         ctypes.c_size_t, _vp, ctypes.c_size_t, _vp]),
    "tfl_kv4_wait_probe": (ctypes.c_int, [_vp, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, ctypes.c_size_t, _vp,
                                          ctypes.c_size_t, ctypes.c_int, ctypes.c_int, _vp]),
    "tfl_kv4_step_workspace_bytes": (ctypes.c_size_t, [_vp]),
    "tfl_decode_step_kv4": (ctypes.c_int, [_vp, _vp, ctypes.POINTER(_vp), ctypes.c_int, _vp, _intp, _vp, _vp,
                                           ctypes.c_size_t, _vp]),
    "tfl_kv4_prompt_workspace_bytes": (ctypes.c_size_t, [_vp, ctypes.c_int]),
    "tfl_prefill_chunk_kv4": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp, ctypes.c_size_t,
                                             _vp]),
    "tfl_beam_select": (ctypes.c_int, [_vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _vp, ctypes.c_int, _vp,
                                       _vp, _vp, _vp, _vp]),
    "tfl_kv_reorder": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp]),
    "tfl_kv_reorder_rows": (ctypes.c_int, [_vp, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp]),
    "tfl_shared_workspace_bytes": (ctypes.c_size_t, [_vp]),
    "tfl_shared_attention": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp,
                                            ctypes.c_size_t, _vp, ctypes.c_size_t, _vp, ctypes.c_size_t, _vp]),
    "tfl_shared_wait_probe": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, ctypes.c_size_t,
                                             _vp, ctypes.c_size_t, _vp, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, _vp]),
    "tfl_decode_step_shared": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
}

_lib = None


def lib():
    """Loads libtfl.so (built by gqa_decoder_forward_gb300.build); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run gqa_decoder_forward_gb300.build.build() first "
                               "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class TflError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{msg} [{code}]")
        self.code = code


def _check(code: int) -> int:
    if code != TFL_OK:
        raise TflError(code, lib().tfl_last_error().decode())
    return code


def _ptr(t) -> int | None:
    if t is None:
        return None
    assert isinstance(t, torch.Tensor) and t.is_contiguous(), "expected a contiguous tensor"
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _settle():
    """Ends the work of the current stream.  The library's objects write into their memory when they are made, in no
    stream's order; a tensor made on the current stream may be the caller's, filled there, or memory that
    earlier work of the stream still uses."""
    torch.cuda.current_stream().synchronize()


def config(shape, max_rows=64, max_decode_rows=64, max_context=4096) -> tfl_config:
    return tfl_config(shape.hidden, shape.layers, shape.n_q, shape.n_kv, shape.head_dim, shape.ffn, shape.vocab,
                      shape.rope_theta, shape.rms_eps, max_rows, max_decode_rows, max_context)


# ---- host-only entry points -------------------------------------------------------

def tfl_qualify(cfg: tfl_config) -> tuple[int, str]:
    buf = ctypes.create_string_buffer(512)
    code = lib().tfl_qualify(ctypes.byref(cfg), buf, 512)
    return code, buf.value.decode()


def tfl_workspace_bytes(cfg: tfl_config) -> int:
    return int(lib().tfl_workspace_bytes(ctypes.byref(cfg)))


def tfl_kv_bytes(cfg: tfl_config, max_positions: int) -> int:
    return int(lib().tfl_kv_bytes(ctypes.byref(cfg), int(max_positions)))


def tfl_rope_table(theta: float, n_pos: int):
    import numpy as np
    c = np.empty((n_pos, 64), np.uint16)
    s = np.empty((n_pos, 64), np.uint16)
    lib().tfl_rope_table(theta, n_pos, c.ctypes.data, s.ctypes.data)
    return c, s


# ---- objects ----------------------------------------------------------------------

class Model:
    """tfl_init over caller-owned weights (dict of bf16 CUDA tensors as made by
    synth.model_weights) plus a workspace tensor this object allocates."""

    def __init__(self, shape, weights: dict, max_rows=64, max_decode_rows=64, max_context=4096):
        self.shape = shape
        self.cfg = config(shape, max_rows, max_decode_rows, max_context)
        self.weights = weights
        nbytes = tfl_workspace_bytes(self.cfg)
        if nbytes == 0:
            code, msg = tfl_qualify(self.cfg)
            raise TflError(code, msg)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        w = tfl_weights()
        w.embed, w.final_norm, w.lm_head = (_ptr(weights[k]) for k in ("embed", "final_norm", "lm_head"))
        self._arrays = {}
        for k in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "wg", "wu", "wd"):
            arr = (_vp * shape.layers)(*[_ptr(t) for t in weights[k]])
            self._arrays[k] = arr
            setattr(w, k, ctypes.cast(arr, ctypes.POINTER(_vp)))
        self._w = w
        h = _vp()
        _settle()
        _check(lib().tfl_init(ctypes.byref(self.cfg), ctypes.byref(w), _ptr(self.workspace), nbytes,
                              ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None):
            lib().tfl_free(self.handle)
            self.handle = None

    def kv(self, max_positions: int) -> "KV":
        return KV(self, max_positions)

    def decode_step(self, kvs: Sequence["KV"], ids: torch.Tensor, rows: Sequence[int], logits: torch.Tensor,
                    stream=None):
        return tfl_decode_step(self, kvs, ids, rows, logits, stream)

    def set_persistent(self, enable: bool):
        """Decode steps of one or two rows as one persistent launch (default) or
        as a launch per operation; the results are bit-identical."""
        return _check(lib().tfl_set_persistent(self.handle, 1 if enable else 0))

    def prefill_chunk(self, kv: "KV", ids: torch.Tensor, logits=None, all_rows=False, stream=None):
        return tfl_prefill_chunk(self, kv, ids, logits, all_rows, stream)

    def argmax(self, logits: torch.Tensor, ids: torch.Tensor, stream=None):
        return tfl_argmax(self, logits, ids, stream)

    def sample(self, logits: torch.Tensor, temperature: float, top_k: int, top_p: float, u: torch.Tensor,
               ids: torch.Tensor, stream=None):
        """Seeded draw per row (u: float32 CUDA tensor of uniforms in [0, 1))."""
        assert u.dtype == torch.float32 and u.is_cuda and ids.dtype == torch.int32
        return _check(lib().tfl_sample(self.handle, _ptr(logits), logits.shape[0], float(temperature), int(top_k),
                                       float(top_p), _ptr(u), _ptr(ids), _stream(stream)))

    def status(self, stream=None) -> int:
        return lib().tfl_status(self.handle, _stream(stream))

    def decode_drafted(self, kv: "KV", context, n_tokens: int, draft_len: int, drafter: "Model" = None,
                       dkv: "KV" = None, stream=None):
        """Drafted greedy decode (tfl_decode_drafted): context = the tokens so far
        (host ints, the last one pending, length(kv) == len(context) - 1).
        Returns (numpy int32 [n_tokens] greedy ids, stats dict)."""
        return tfl_decode_drafted(self, kv, context, n_tokens, draft_len, drafter, dkv, stream)


class KV:
    """A paged bf16 cache (tfl_kv) over `buffer` (a uint8 CUDA tensor of at least tfl_kv_bytes bytes, whose
    pages are kept; work on it may be queued on the current stream) or one that it allocates."""

    def __init__(self, model: Model, max_positions: int, buffer: torch.Tensor = None):
        self.model = model
        nbytes = tfl_kv_bytes(model.cfg, max_positions)
        device = _device_of(model)
        if device != torch.cuda.current_device():
            raise ValueError(f"the model is on device {device} and the current device is {torch.cuda.current_device()}")
        if buffer is None:
            buffer = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        if not buffer.is_cuda or not buffer.is_contiguous() or buffer.get_device() != device:
            raise ValueError(f"expected a contiguous buffer on the model's device, got strides {buffer.stride()} on {buffer.device}")
        self.buffer = buffer
        h = _vp()
        _settle()
        _check(lib().tfl_kv_alloc(model.handle, int(max_positions), _ptr(buffer),
                                  buffer.numel() * buffer.element_size(), ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None):
            lib().tfl_kv_free(self.handle)
            self.handle = None

    @property
    def length(self) -> int:
        return int(lib().tfl_kv_length(self.handle))

    def reset(self, keep: int):
        _check(lib().tfl_kv_reset(self.handle, int(keep)))

    def write(self, layer: int, pos0: int, k: torch.Tensor, v: torch.Tensor, stream=None):
        _check(lib().tfl_kv_write(self.model.handle, self.handle, layer, pos0, k.shape[0], _ptr(k), _ptr(v),
                                  _stream(stream)))

    def read(self, layer: int, pos0: int, n: int, stream=None):
        s = self.model.shape
        k = torch.empty((n, s.n_kv, s.head_dim), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        _check(lib().tfl_kv_read(self.model.handle, self.handle, layer, pos0, n, _ptr(k), _ptr(v),
                                 _stream(stream)))
        return k, v


# ---- device entry points (C names) --------------------------------------------------

def _kv_array(kvs):
    return (_vp * len(kvs))(*[kv.handle for kv in kvs])


def tfl_decode_step(model: Model, kvs, ids, rows, logits, stream=None):
    assert ids.dtype == torch.int32 and logits.dtype == torch.bfloat16
    r = (ctypes.c_int * len(rows))(*rows)
    return _check(lib().tfl_decode_step(model.handle, _kv_array(kvs), len(kvs), _ptr(ids), r, _ptr(logits),
                                        _stream(stream)))


def tfl_decode_hidden(model: Model, kvs, rows, h_in, h_out, stream=None):
    r = (ctypes.c_int * len(rows))(*rows)
    return _check(lib().tfl_decode_hidden(model.handle, _kv_array(kvs), len(kvs), r, _ptr(h_in), _ptr(h_out),
                                          _stream(stream)))


def tfl_prefill_chunk(model: Model, kv: KV, ids, logits=None, all_rows=False, stream=None):
    assert ids.dtype == torch.int32
    return _check(lib().tfl_prefill_chunk(model.handle, kv.handle, _ptr(ids), ids.numel(), _ptr(logits),
                                          1 if all_rows else 0, _stream(stream)))


def tfl_prefill_hidden(model: Model, kv: KV, h_in, h_out, stream=None):
    return _check(lib().tfl_prefill_hidden(model.handle, kv.handle, _ptr(h_in), h_in.shape[0], _ptr(h_out),
                                           _stream(stream)))


def tfl_head(model: Model, h, logits, stream=None):
    return _check(lib().tfl_head(model.handle, _ptr(h), h.shape[0], _ptr(logits), _stream(stream)))


def tfl_argmax(model: Model, logits, ids, stream=None):
    return _check(lib().tfl_argmax(model.handle, _ptr(logits), logits.shape[0], _ptr(ids), _stream(stream)))


def tfl_status(model: Model, stream=None) -> int:
    return int(lib().tfl_status(model.handle, _stream(stream)))


def tfl_wait_probe(model: Model, which: int, spin_limit: int, stream=None):
    """Runs one bounded device wait (0: grid barrier, 1: mbarrier) on an event
    that never happens; tfl_status then reports TFL_E_DEVICE."""
    return _check(lib().tfl_wait_probe(model.handle, int(which), int(spin_limit), _stream(stream)))


TFL_OP_PROMPT = 0x100
OPS = {"attn_norm": 0, "qkv_rope": 1, "attention": 2, "o_residual": 3, "ffn_norm": 4, "gate_up": 5,
       "down_residual": 6, "final_norm": 7, "lm_head": 8, "norm_qkv_rope": 9, "norm_gate_up": 10,
       "norm_lm_head": 11}


def tfl_layer_op(model: Model, op: str, layer: int, inp: torch.Tensor, out: torch.Tensor, kv: "KV" = None,
                 pos0: int = 0, stream=None, prompt: bool = False):
    """One op of the decode path (prompt=True: of the prompt-chunk path)."""
    code = OPS[op] | (TFL_OP_PROMPT if prompt else 0)
    return _check(lib().tfl_layer_op(model.handle, code, layer, kv.handle if kv is not None else None, pos0,
                                     inp.shape[0], _ptr(inp), _ptr(out), _stream(stream)))


def tfl_attention_decode_noalloc(kv: "KV", layer: int, pos0: int, q: torch.Tensor, out: torch.Tensor, stream=None):
    """Decode attention with the library's fixed scratch (no allocation, no workspace)."""
    return _check(lib().tfl_attention_decode_noalloc(kv.handle, layer, pos0, q.shape[0], _ptr(q), _ptr(out),
                                                     _stream(stream)))


def tfl_profile(model: Model, enable: bool):
    return _check(lib().tfl_profile(model.handle, 1 if enable else 0))


def tfl_kv_copy_prefix(model: Model, src: "KV", dst: "KV", n: int, stream=None):
    """Copies positions [0, n) of every layer from src to dst; length(dst) = n."""
    _check(lib().tfl_kv_copy_prefix(model.handle, src.handle, dst.handle, n, _stream(stream)))


class PrefixStore:
    """Host index of caches holding prompt prefixes (tfl_prefix_store_*); the
    caches stay owned by the caller (KV objects are kept referenced here)."""

    def __init__(self, max_entries: int):
        h = _vp()
        _check(lib().tfl_prefix_store_new(max_entries, ctypes.byref(h)))
        self.handle = h
        self._kvs = {}

    def __del__(self):
        if getattr(self, "handle", None):
            lib().tfl_prefix_store_free(self.handle)
            self.handle = None

    @staticmethod
    def _tok(tokens):
        t = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        return t, t.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))

    def put(self, tokens, kv: "KV"):
        t, p = self._tok(tokens)
        _check(lib().tfl_prefix_store_put(self.handle, p, len(t), kv.handle))
        self._kvs[kv.handle.value if hasattr(kv.handle, "value") else kv.handle] = kv

    def match(self, tokens):
        """(KV or None, matched token count)."""
        t, p = self._tok(tokens)
        h, n = _vp(), ctypes.c_int()
        _check(lib().tfl_prefix_store_match(self.handle, p, len(t), ctypes.byref(h), ctypes.byref(n)))
        return (self._kvs.get(h.value) if h.value else None), n.value

    def remove(self, kv: "KV"):
        _check(lib().tfl_prefix_store_remove(self.handle, kv.handle))
        self._kvs.pop(kv.handle.value if hasattr(kv.handle, "value") else kv.handle, None)

    def __len__(self):
        return lib().tfl_prefix_store_size(self.handle)


def tfl_copy_draft(tokens, max_draft: int) -> np.ndarray:
    """Copy-draft guesses for the tokens so far (host only)."""
    t = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
    out = np.zeros(max(max_draft, 1), np.int32)
    n = _check_count(lib().tfl_copy_draft(t.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), len(t), int(max_draft),
                                          out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))))
    return out[:n]


def _check_count(code: int) -> int:
    if code < 0:
        raise TflError(code, lib().tfl_last_error().decode())
    return code


def tfl_decode_drafted(model: Model, kv: KV, context, n_tokens: int, draft_len: int, drafter: Model = None,
                       dkv: KV = None, stream=None):
    ctx = np.ascontiguousarray(np.asarray(context, dtype=np.int32))
    out = np.full(int(n_tokens), -1, np.int32)
    nbytes = int(lib().tfl_drafted_workspace_bytes(model.handle, int(draft_len)))
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
    st = tfl_draft_stats()
    i32 = ctypes.POINTER(ctypes.c_int32)
    code = lib().tfl_decode_drafted(model.handle, kv.handle, drafter.handle if drafter is not None else None,
                                    dkv.handle if dkv is not None else None, int(draft_len),
                                    ctx.ctypes.data_as(i32), len(ctx), int(n_tokens), out.ctypes.data_as(i32),
                                    _ptr(ws), nbytes, ctypes.byref(st), _stream(stream))
    stats = {k: int(getattr(st, k)) for k, _ in tfl_draft_stats._fields_}
    if code != TFL_OK:
        err = TflError(code, lib().tfl_last_error().decode())
        err.ids, err.stats = out, stats
        raise err
    return out, stats


STEP_PHASES = ("qkv", "attention", "merge", "o", "gate_up", "down", "barrier", "head", "total")


def tfl_step_phases(model: Model) -> dict:
    """{phase: microseconds} of the last persistent decode step run while profiling."""
    out = (ctypes.c_double * len(STEP_PHASES))()
    _check(lib().tfl_step_phases(model.handle, out, len(STEP_PHASES)))
    return {k: round(v, 3) for k, v in zip(STEP_PHASES, out)}


def tfl_profile_read(model: Model) -> dict:
    """{family name: (total ms, launches)} recorded since the last read."""
    names = []
    while True:
        n = lib().tfl_profile_kind(len(names))
        if n is None:
            break
        names.append(n.decode())
    ms = (ctypes.c_double * len(names))()
    cnt = (ctypes.c_long * len(names))()
    _check(lib().tfl_profile_read(model.handle, len(names), ms, cnt))
    return {names[i]: (ms[i], cnt[i]) for i in range(len(names))}


# ---- 4-bit KV cache -----------------------------------------------------------------

def tfl_kv4_bytes(layers: int, n_kv: int, max_positions: int, head_dim: int = 128) -> int:
    return int(lib().tfl_kv4_bytes(layers, n_kv, head_dim, max_positions))


class KV4:
    """A paged cache in 4 bits (tfl_kv4) over `buffer` (a uint8 CUDA tensor of at
    least tfl_kv4_bytes bytes, whose contents are kept; work on it may be queued on the
    current stream) or one that it allocates.  Outlives the calls on other streams than
    the one it was made on."""

    def __init__(self, layers: int, n_kv: int, max_positions: int, buffer: torch.Tensor = None):
        nbytes = tfl_kv4_bytes(layers, n_kv, max_positions)
        if buffer is None:
            buffer = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        if not buffer.is_cuda or not buffer.is_contiguous() or buffer.get_device() != torch.cuda.current_device():
            raise ValueError(f"expected a contiguous buffer on the current device, got strides {buffer.stride()} on {buffer.device}")
        self.layers, self.n_kv, self.buffer = layers, n_kv, buffer
        h = _vp()
        _settle()
        _check(lib().tfl_kv4_alloc(layers, n_kv, 128, int(max_positions), _ptr(buffer),
                                   buffer.numel() * buffer.element_size(), ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None):
            lib().tfl_kv4_free(self.handle)
            self.handle = None

    @property
    def length(self) -> int:
        return int(lib().tfl_kv4_length(self.handle))

    @property
    def capacity(self) -> int:
        return int(lib().tfl_kv4_capacity(self.handle))

    def reset(self, keep: int):
        _check(lib().tfl_kv4_reset(self.handle, int(keep)))


class KV4Rows:
    """Rows of a call over 4-bit caches: stream s has rows[s] rows at positions
    pos0[s] on.  Keeps the host arrays that the library takes, so that a step's
    layers (and, with set, its successors) make them once."""

    def __init__(self, kvs: Sequence[KV4], pos0: Sequence[int], rows: Sequence[int]):
        self.kvs = list(kvs)
        self.n = len(self.kvs)
        self.device = self.kvs[0].buffer.get_device() if self.kvs else -1
        self.handles = (_vp * self.n)(*[kv.handle for kv in self.kvs])
        self.pos0 = (ctypes.c_int * self.n)()
        self.rows = (ctypes.c_int * self.n)()
        self.handles_at, self.pos0_at, self.rows_at = map(ctypes.addressof, (self.handles, self.pos0, self.rows))
        self.set(pos0, rows)

    def set(self, pos0: Sequence[int], rows: Sequence[int]):
        if len(pos0) != self.n or len(rows) != self.n:
            raise ValueError(f"{len(pos0)} positions and {len(rows)} row counts for {self.n} caches")
        pos0, rows = list(map(operator.index, pos0)), list(map(operator.index, rows))
        if not all(-2 ** 31 <= x < 2 ** 31 for x in pos0 + rows):  # an int array would keep their low halves
            raise ValueError(f"positions {pos0} or row counts {rows} outside 32 bits")
        self.pos0[:] = pos0
        self.rows[:] = rows
        self.total = sum(rows)
        self.n_kv = self.kvs[0].n_kv if self.kvs else 0


class KV4Attention:
    """tfl_kv4_attn and its workspace: attention of up to max_rows rows over caches
    of up to max_positions positions.  Outlives the calls on other streams than the one
    it was made on."""

    def __init__(self, n_q: int, n_kv: int, max_rows: int = 16, max_positions: int = 4096):
        nbytes = int(lib().tfl_kv4_attn_bytes(n_q, n_kv, 128, max_rows, max_positions))
        self.n_q, self.n_kv = n_q, n_kv
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
        h = _vp()
        _settle()
        _check(lib().tfl_kv4_attn_init(n_q, n_kv, 128, max_rows, max_positions, _ptr(self.workspace), nbytes,
                                       ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None):
            lib().tfl_kv4_attn_free(self.handle)
            self.handle = None


def tfl_kv4_attn_status(attn: KV4Attention, stream=None) -> int:
    return int(lib().tfl_kv4_attn_status(attn.handle, _stream(stream)))


def _rows_arg(t: torch.Tensor, batch: KV4Rows, heads: int) -> int:
    """Row stride (elements) of a bf16 CUDA tensor, on the caches' device, of at least the
    batch's rows of heads x 128 numbers, [rows, heads, 128] or [rows, heads * 128]; only rows may be strided."""
    if t.dtype is not torch.bfloat16 or not t.is_cuda or t.get_device() != batch.device:
        raise ValueError(f"expected a bf16 tensor on CUDA device {batch.device}")
    n = batch.total
    if n == 0:
        return heads * 128  # nothing is read or written: whatever the shape
    sh, st = t.shape, t.stride()
    if len(sh) == 2:
        ok = sh[1] == heads * 128 and st[1] == 1
    else:
        ok = len(sh) == 3 and sh[1] == heads and sh[2] == 128 and st[2] == 1 and (heads == 1 or st[1] == 128)
    if not ok or sh[0] < n:
        raise ValueError(f"expected [>= {n}, {heads} * 128] with contiguous rows, got {tuple(sh)} strides {st}")
    return st[0] if n > 1 else heads * 128  # of one row, whatever its tensor's stride


def _stream_of(t: torch.Tensor, stream) -> int:
    """The stream to enqueue on: torch's current one of the tensor's device if none is given (looked up without
    making a Stream object, which would cost as much as a launch)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else _stream(stream)


def tfl_kv4_write(batch: KV4Rows, layer: int, k: torch.Tensor, v: torch.Tensor, stream=None):
    """Quantises rows k, v into the caches of batch."""
    ld = _rows_arg(k, batch, batch.n_kv)
    if _rows_arg(v, batch, batch.n_kv) != ld:
        raise ValueError("k and v have different row strides")
    return _check(lib().tfl_kv4_write(batch.handles_at, batch.n, layer, batch.pos0_at, batch.rows_at, k.data_ptr(),
                                      v.data_ptr(), ld, _stream_of(k, stream)))


def tfl_kv4_read(batch: KV4Rows, layer: int, k: torch.Tensor, v: torch.Tensor, stream=None):
    """Reads what the caches of batch stand for into k, v."""
    ld = _rows_arg(k, batch, batch.n_kv)
    if _rows_arg(v, batch, batch.n_kv) != ld:
        raise ValueError("k and v have different row strides")
    return _check(lib().tfl_kv4_read(batch.handles_at, batch.n, layer, batch.pos0_at, batch.rows_at, k.data_ptr(),
                                     v.data_ptr(), ld, _stream_of(k, stream)))


def tfl_kv4_attention(attn: KV4Attention, batch: KV4Rows, layer: int, q: torch.Tensor, out: torch.Tensor,
                      stream=None):
    """Attention of the rows q over the caches of batch (which hold those rows' own keys and values)."""
    ldq = _rows_arg(q, batch, attn.n_q)
    ldo = _rows_arg(out, batch, attn.n_q)
    return _check(lib().tfl_kv4_attention(attn.handle, batch.handles_at, batch.n, layer, batch.pos0_at, batch.rows_at,
                                          q.data_ptr(), ldq, out.data_ptr(), ldo, _stream_of(q, stream)))


def tfl_kv4_wait_probe(attn: KV4Attention, batch: KV4Rows, layer: int, q: torch.Tensor, out: torch.Tensor, lose: int,
                       spin_limit: int, stream=None):
    """tfl_kv4_attention with a copy that never comes: tfl_kv4_attn_status then reports TFL_E_DEVICE."""
    ldq = _rows_arg(q, batch, attn.n_q)
    ldo = _rows_arg(out, batch, attn.n_q)
    return _check(lib().tfl_kv4_wait_probe(attn.handle, batch.handles_at, batch.n, layer, batch.pos0_at, batch.rows_at,
                                           q.data_ptr(), ldq, out.data_ptr(), ldo, lose, spin_limit,
                                           _stream_of(q, stream)))


class KV4Runner:
    """The forward of a model over 4-bit caches: the attention object and the
    workspaces of tfl_decode_step_kv4 (up to max_rows rows) and tfl_prefill_chunk_kv4,
    for caches of up to max_positions positions.  One call at a time."""

    def __init__(self, model: Model, max_rows: int = 16, max_positions: int = 4096):
        s = model.shape
        self.model = model
        self.max_positions = max_positions
        self.attention = KV4Attention(s.n_q, s.n_kv, max_rows, max_positions)
        self.step_ws = torch.empty(int(lib().tfl_kv4_step_workspace_bytes(model.handle)), dtype=torch.uint8,
                                   device="cuda")
        # a model's prompts end at its max_context, whatever the caches hold
        self.prompt_ws = torch.empty(
            int(lib().tfl_kv4_prompt_workspace_bytes(model.handle, min(max_positions, model.cfg.max_context))),
            dtype=torch.uint8, device="cuda")

    def kv(self, max_positions: int) -> KV4:
        return KV4(self.model.shape.layers, self.model.shape.n_kv, max_positions)

    def decode_step(self, kvs: Sequence[KV4], ids: torch.Tensor, rows: Sequence[int], logits: torch.Tensor,
                    stream=None):
        return tfl_decode_step_kv4(self, kvs, ids, rows, logits, stream)

    def prefill_chunk(self, kv: KV4, ids: torch.Tensor, logits=None, all_rows=False, stream=None):
        return tfl_prefill_chunk_kv4(self, kv, ids, logits, all_rows, stream)


def _check_ids_and_logits(runner: KV4Runner, ids, logits, n: int, rows: int):
    """At least n int32 ids, and bf16 logits (or None) for at least so many rows, on the runner's device."""
    vocab = runner.model.shape.vocab
    for t in (ids, logits):
        if t is not None and t.get_device() != runner.step_ws.get_device():
            raise ValueError(f"expected ids and logits on {runner.step_ws.device}, got {t.device}")
    if ids.dtype != torch.int32 or ids.numel() < n:
        raise ValueError(f"expected {n} int32 ids, got {ids.numel()} of {ids.dtype}")
    if logits is not None and (logits.dtype != torch.bfloat16 or logits.numel() < rows * vocab):
        raise ValueError(f"expected bf16 logits of {rows} rows of {vocab}, got {tuple(logits.shape)} of {logits.dtype}")


def tfl_decode_step_kv4(runner: KV4Runner, kvs, ids, rows, logits, stream=None):
    """tfl_decode_step over 4-bit caches: rows[s] ids of each cache, one after the other, to as many rows of logits."""
    if len(rows) != len(kvs):
        raise ValueError(f"{len(rows)} row counts for {len(kvs)} caches")
    _check_ids_and_logits(runner, ids, logits, sum(rows), sum(rows))
    r = (ctypes.c_int * len(rows))(*rows)
    return _check(lib().tfl_decode_step_kv4(runner.model.handle, runner.attention.handle, _kv_array(kvs), len(kvs),
                                            _ptr(ids), r, _ptr(logits), _ptr(runner.step_ws), runner.step_ws.numel(),
                                            _stream(stream)))


def tfl_prefill_chunk_kv4(runner: KV4Runner, kv: KV4, ids, logits=None, all_rows=False, stream=None):
    """tfl_prefill_chunk into a 4-bit cache; logits: None, or of the last row, or of all rows."""
    _check_ids_and_logits(runner, ids, logits, 1, ids.numel() if all_rows else 1)
    return _check(lib().tfl_prefill_chunk_kv4(runner.model.handle, kv.handle, _ptr(ids), ids.numel(), _ptr(logits),
                                              1 if all_rows else 0, _ptr(runner.prompt_ws), runner.prompt_ws.numel(),
                                              _stream(stream)))


# ---- several continuations of one prompt -------------------------------------------------

def _ints(values, n: int, what: str):
    """A C int array of n values, which must fit it (an int array would keep their low halves)."""
    values = list(map(operator.index, values))
    if len(values) != n:
        raise ValueError(f"{len(values)} {what}, expected {n}")
    if not all(-2 ** 31 <= x < 2 ** 31 for x in values):
        raise ValueError(f"{what} {values} outside 32 bits")
    return (ctypes.c_int * n)(*values)


def _int32(x: int, what: str) -> int:
    """x, which becomes a C int."""
    if -2 ** 31 <= x < 2 ** 31:
        return x
    raise ValueError(f"{what} {x} outside 32 bits")


def _device_of(model: Model) -> int:
    return model.workspace.get_device()


def _vector(t: torch.Tensor, dtype, shape: tuple, device: int, what: str) -> int:
    """Address of a contiguous CUDA tensor of this type, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    raise ValueError(f"{what}: expected contiguous {dtype} {shape} on CUDA device {device}, got {t.dtype} "
                     f"{tuple(t.shape)} strides {t.stride()} on {t.device}")


def tfl_beam_select(model: Model, logits: torch.Tensor, scores: torch.Tensor, ids: torch.Tensor, parents: torch.Tensor,
                    out_scores: torch.Tensor, eos: int = -1, done: torch.Tensor = None, out_done: torch.Tensor = None,
                    stream=None):
    """The best continuations of each group's beams: logits [groups * beams, V] bf16, scores [groups, beams] float32 (and
    done, int32) in; ids, parents (rows of logits) int32, out_scores float32 (and out_done, int32) [groups, n_out] out."""
    if len(scores.shape) != 2 or len(ids.shape) != 2:
        raise ValueError(f"expected scores [groups, beams] and ids [groups, n_out], got {tuple(scores.shape)} and {tuple(ids.shape)}")
    dev = model.workspace.get_device()
    groups, beams = given = tuple(scores.shape)
    n_out = ids.shape[1]
    out, i32, f32 = (groups, n_out), torch.int32, torch.float32
    return _check(lib().tfl_beam_select(
        model.handle, _vector(logits, torch.bfloat16, (groups * beams, model.shape.vocab), dev, "logits"), groups, beams, n_out,
        _vector(scores, f32, given, dev, "scores"), None if done is None else _vector(done, i32, given, dev, "done"),
        _int32(eos, "eos"),
        _vector(ids, i32, out, dev, "ids"), _vector(parents, i32, out, dev, "parents"),
        _vector(out_scores, f32, out, dev, "out_scores"),
        None if out_done is None else _vector(out_done, i32, out, dev, "out_done"), _stream_of(logits, stream)))


class KVRows:
    """Ranges of bf16 caches: positions pos0[i] .. pos0[i] + rows[i] - 1 of kvs[i].  Keeps the host arrays that the
    library takes, so that a search's steps make the caches' once (set: other ranges)."""

    def __init__(self, kvs: Sequence[KV], pos0: Sequence[int], rows: Sequence[int]):
        self.kvs = list(kvs)
        self.n = len(self.kvs)
        self.handles = _kv_array(self.kvs)
        self.set(pos0, rows)

    def set(self, pos0: Sequence[int], rows: Sequence[int]):
        pos0, rows = _ints(pos0, self.n, "positions"), _ints(rows, self.n, "row counts")
        self.pos0, self.rows = pos0, rows


def _parents(model: Model, batch: KVRows, parents: torch.Tensor) -> int:
    if parents.dtype is not torch.int32 or parents.get_device() != _device_of(model) or parents.numel() != batch.n \
            or not parents.is_contiguous():
        raise ValueError(f"expected {batch.n} contiguous int32 parents on CUDA device {_device_of(model)}, got "
                         f"{parents.dtype} {tuple(parents.shape)} strides {parents.stride()} on {parents.device}")
    return parents.data_ptr()


def tfl_kv_reorder(model: Model, batch: KVRows, parents: torch.Tensor, stream=None):
    """The ranges of batch take what the caches numbered by parents (int32, one per cache) hold there."""
    return _check(lib().tfl_kv_reorder(model.handle, batch.handles, batch.n, batch.pos0, batch.rows,
                                       _parents(model, batch, parents), _stream_of(parents, stream)))


def tfl_kv_reorder_rows(model: Model, batch: KVRows, first: int, parents: torch.Tensor, stream=None):
    """tfl_kv_reorder where batch's caches are those of rows first .. first + n - 1 of a larger call, which parents number
    (the group's row of a selection's parents)."""
    return _check(lib().tfl_kv_reorder_rows(model.handle, batch.handles, batch.n, _int32(first, "first row"), batch.pos0,
                                            batch.rows, _parents(model, batch, parents), _stream_of(parents, stream)))


class SharedRows:
    """Streams over shared prefixes: group g's streams[g] streams, each with a cache of tails, share prefixes[g] (None:
    no prefix); n_prefix[g] positions of it (default: its length now; a decode step takes whole prefixes, as long as they are
    here); stream s's row at position pos[s] (needed for tfl_shared_attention alone).  Keeps the host arrays that the library
    takes (set: other positions)."""

    def __init__(self, prefixes: Sequence[KV], streams: Sequence[int], tails: Sequence[KV], n_prefix: Sequence[int] = None,
                 pos: Sequence[int] = None):
        self.prefixes, self.tails = list(prefixes), list(tails)
        self.n_groups = len(self.prefixes)
        self.streams = _ints(streams, self.n_groups, "stream counts")
        if sum(self.streams) != len(self.tails):
            raise ValueError(f"{len(self.tails)} tails for groups of {list(self.streams)} streams")
        self.prefix_handles = (_vp * self.n_groups)(*[None if kv is None else kv.handle for kv in self.prefixes])
        self.tail_handles = _kv_array(self.tails)
        if n_prefix is None:
            n_prefix = [0 if kv is None else kv.length for kv in self.prefixes]
        self.n_prefix = _ints(n_prefix, self.n_groups, "prefix lengths")
        self.pos = None
        if pos is not None:
            self.set(pos)

    def set(self, pos: Sequence[int]):
        self.pos = _ints(pos, len(self.tails), "positions")


class SharedRunner:
    """The workspace of tfl_shared_attention and tfl_decode_step_shared.  One call at a time."""

    def __init__(self, model: Model):
        self.model = model
        self.workspace = torch.empty(int(lib().tfl_shared_workspace_bytes(model.handle)), dtype=torch.uint8,
                                     device=model.workspace.device)

    def decode_step(self, batch: SharedRows, ids: torch.Tensor, logits: torch.Tensor, stream=None):
        return tfl_decode_step_shared(self, batch, ids, logits, stream)


def _head_rows(t: torch.Tensor, model: Model, n: int, what: str) -> int:
    """Row stride (elements) of a bf16 tensor [>= n, n_q * 128] or [>= n, n_q, 128]; only rows may be strided."""
    heads, sh, st = model.shape.n_q, t.shape, t.stride()
    if len(sh) == 2:
        ok = sh[1] == heads * 128 and st[1] == 1
    else:
        ok = len(sh) == 3 and tuple(sh[1:]) == (heads, 128) and st[1:] == (128, 1)
    if not ok or sh[0] < n or t.dtype is not torch.bfloat16 or t.get_device() != _device_of(model):
        raise ValueError(f"{what}: expected bf16 [>= {n}, {heads} * 128] with contiguous rows on CUDA device "
                         f"{_device_of(model)}, got {t.dtype} {tuple(sh)} strides {st} on {t.device}")
    return st[0] if n > 1 else heads * 128  # of one row, whatever its tensor's stride


def _shared_args(runner: SharedRunner, batch: SharedRows, layer: int, q: torch.Tensor, out: torch.Tensor):
    if batch.pos is None:
        raise ValueError("the batch has no positions")
    m, n, ws = runner.model, len(batch.tails), runner.workspace
    ldq, ldo = _head_rows(q, m, n, "q"), _head_rows(out, m, n, "out")
    return (m.handle, _int32(layer, "layer"), batch.prefix_handles, batch.n_prefix, batch.streams, batch.n_groups, batch.tail_handles, batch.pos,
            q.data_ptr(), ldq, out.data_ptr(), ldo, ws.data_ptr(), ws.numel())


def tfl_shared_attention(runner: SharedRunner, batch: SharedRows, layer: int, q: torch.Tensor, out: torch.Tensor, stream=None):
    """Attention of one row per stream over its group's prefix and its own tail."""
    return _check(lib().tfl_shared_attention(*_shared_args(runner, batch, layer, q, out), _stream_of(q, stream)))


def tfl_shared_wait_probe(runner: SharedRunner, batch: SharedRows, layer: int, q: torch.Tensor, out: torch.Tensor, lose: int,
                          spin_limit: int, stream=None):
    """tfl_shared_attention with a loader that stops at keys (2 k) or values (2 k + 1) of block k: tfl_status then reports
    TFL_E_DEVICE."""
    return _check(lib().tfl_shared_wait_probe(*_shared_args(runner, batch, layer, q, out), _int32(lose, "lose"),
                                              _int32(spin_limit, "spin_limit"), _stream_of(q, stream)))


def tfl_decode_step_shared(runner: SharedRunner, batch: SharedRows, ids: torch.Tensor, logits: torch.Tensor, stream=None):
    """tfl_decode_step of one id per stream, over shared prefixes; the caches' lengths say where the rows sit, and the prefixes' have
    to be the batch's, which its tails were made for."""
    m, n = runner.model, len(batch.tails)
    for g, kv in enumerate(batch.prefixes):
        length = 0 if kv is None else kv.length
        if batch.n_prefix[g] != length:
            raise ValueError(f"group {g}: a batch for {batch.n_prefix[g]} positions of a prefix whose length is {length}")
    if ids.dtype is not torch.int32 or ids.get_device() != _device_of(m) or ids.numel() != n or not ids.is_contiguous():
        raise ValueError(f"expected {n} contiguous int32 ids on CUDA device {_device_of(m)}, got {ids.dtype} "
                         f"{tuple(ids.shape)} strides {ids.stride()} on {ids.device}")
    return _check(lib().tfl_decode_step_shared(m.handle, batch.prefix_handles, batch.streams, batch.n_groups,
                                               batch.tail_handles, ids.data_ptr(),
                                               _vector(logits, torch.bfloat16, (n, m.shape.vocab), _device_of(m), "logits"),
                                               runner.workspace.data_ptr(), runner.workspace.numel(),
                                               _stream_of(ids, stream)))
