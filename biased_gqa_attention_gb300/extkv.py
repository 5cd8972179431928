"""Thin ctypes binding over libextkv (include/extkv.h).

Argument marshalling only: torch tensors supply device memory and the current
CUDA stream; every step of the path runs in the library's kernels.  There is
no fallback: if libextkv.so is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libextkv.so")

EXTKV_F32, EXTKV_BF16 = 0, 1
EXTKV_OK, EXTKV_ERR_INVALID_ARG, EXTKV_ERR_UNSUPPORTED, EXTKV_ERR_CUDA, EXTKV_ERR_DEVICE = 0, -1, -2, -3, -4
EXTKV_DEV_BAD_WRITE_IDX, EXTKV_DEV_BAD_NONPAD, EXTKV_DEV_TIMEOUT, EXTKV_DEV_BOUNDS = 0x1, 0x2, 0x4, 0x8
EXTKV_DEV_BAD_PAGE, EXTKV_DEV_BAD_SEQLENS = 0x10, 0x20
ALGO_AUTO, ALGO_GENERIC, ALGO_DECODE, ALGO_PREFILL, ALGO_PREFILL_PAIR = 0, 1, 2, 3, 4
ALGO_DECODE_STREAMK, ALGO_DECODE_CLUSTER = 5, 6

# Every symbol include/extkv.h declares.
SYMBOLS = ("ext_kv_scatter", "build_static_cache_bias", "attention_ext_kv_workspace_size",
           "attention_ext_kv", "attention_ext_kv_scatter", "attention_ext_kv_softcap",
           "build_bias_from_bool_mask", "attention_ext_kv_dv", "attention_ext_kv_workspace_size_dv",
           "extkv_clear_status", "extkv_read_status",
           "extkv_last_error", "extkv_last_kernel", "extkv_last_launches", "extkv_set_algo",
           "extkv_set_wait_polls",
           "attention_ext_kv_noalloc",
           "extkv_step_begin", "extkv_step_end", "extkv_step_launch", "extkv_step_free",
           "rotary_multi_axis", "paged_kv_append", "attention_paged_decode",
           "attention_paged_decode_workspace_size", "attention_packed_prefill",
           "attention_packed_prefill_workspace_size")


class ExtKVError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"extkv error {code}: {message}")
        self.code = code


class _Rotary(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p)]


class _BiasSpec(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("span_offsets", ctypes.c_void_p), ("spans", ctypes.c_void_p),
                ("extra", ctypes.c_void_p), ("q_start", ctypes.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libextkv.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with biased_gqa_attention_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I64, I, I32P = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.ext_kv_scatter.argtypes = [P, P, P, P, P, I64, I64, I64, I64, I64, I, I32P, P]
    lib.build_static_cache_bias.argtypes = [P, ctypes.POINTER(_BiasSpec), P, I64, I64, I64, I, I32P, P]
    lib.build_bias_from_bool_mask.argtypes = [P, P, I64, I64, I64, I, P]
    lib.attention_ext_kv_softcap.argtypes = [P, P, P, P, P, ctypes.POINTER(_BiasSpec), P, ctypes.c_float,
                                             ctypes.c_float, I64, I64, I64, I64, I64, I64, I, P, ctypes.c_size_t,
                                             I32P, P]
    lib.attention_ext_kv_workspace_size.argtypes = [I64, I64, I64, I64, I64, I64, I]
    lib.attention_ext_kv_workspace_size.restype = ctypes.c_size_t
    lib.attention_ext_kv_workspace_size_dv.argtypes = [I64, I64, I64, I64, I64, I64, I64, I]
    lib.attention_ext_kv_workspace_size_dv.restype = ctypes.c_size_t
    lib.attention_ext_kv_dv.argtypes = [P, P, P, P, P, ctypes.POINTER(_BiasSpec), P, ctypes.c_float,
                                        ctypes.c_float, I64, I64, I64, I64, I64, I64, I64, I, P, ctypes.c_size_t,
                                        I32P, P]
    lib.attention_ext_kv.argtypes = [P, P, P, P, P, ctypes.POINTER(_BiasSpec), P, ctypes.c_float,
                                     I64, I64, I64, I64, I64, I64, I, P, ctypes.c_size_t, I32P, P]
    lib.attention_ext_kv_scatter.argtypes = [P, P, P, P, P, P, P, I64, P, ctypes.POINTER(_BiasSpec), P,
                                             ctypes.c_float, I64, I64, I64, I64, I64, I64, I, P,
                                             ctypes.c_size_t, I32P, P]
    lib.attention_ext_kv_noalloc.argtypes = [P, P, P, P, P, ctypes.POINTER(_BiasSpec), P,
                                             ctypes.c_float, I64, I64, I64, I64, I64, I64, I, I32P, P]
    lib.extkv_clear_status.argtypes = [I32P, P]
    lib.extkv_read_status.argtypes = [I32P, P]
    lib.extkv_last_error.restype = ctypes.c_char_p
    lib.extkv_last_kernel.restype = ctypes.c_char_p
    lib.extkv_last_launches.restype = ctypes.c_int
    lib.extkv_set_algo.argtypes = [I]
    lib.extkv_set_wait_polls.argtypes = [I]
    lib.extkv_set_wait_polls.restype = I
    lib.extkv_step_begin.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
    lib.extkv_step_begin.restype = I
    lib.extkv_step_end.argtypes = [P, ctypes.POINTER(ctypes.c_void_p)]
    lib.extkv_step_end.restype = I
    lib.extkv_step_launch.argtypes = [P, P]
    lib.extkv_step_launch.restype = I
    lib.extkv_step_free.argtypes = [P]
    lib.extkv_step_free.restype = None
    I32, F, SZ, ROT = ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(_Rotary)
    lib.rotary_multi_axis.argtypes = [P, P, P, P, ROT, I64, I64, I64, I64, I64, I, P]
    lib.paged_kv_append.argtypes = [P, P, P, P, P, P, P, P, P, ROT] + [I64] * 11 + [I, I32P, P]
    lib.attention_paged_decode.argtypes = [P, P, P, P, P, P, F, I32] + [I64] * 8 + [I, P, SZ, I32P, P]
    lib.attention_paged_decode_workspace_size.argtypes = [I64, I64, I64, I64, I]
    lib.attention_paged_decode_workspace_size.restype = SZ
    lib.attention_packed_prefill.argtypes = [P, P, P, P, P, F, I32, I32] + [I64] * 8 + [I, P, SZ, I32P, P]
    lib.attention_packed_prefill_workspace_size.argtypes = [I64, I64, I64, I64, I64, I]
    lib.attention_packed_prefill_workspace_size.restype = SZ
    for name in ("rotary_multi_axis", "paged_kv_append", "attention_paged_decode", "attention_packed_prefill"):
        getattr(lib, name).restype = I
    for name in ("ext_kv_scatter", "build_static_cache_bias", "attention_ext_kv", "attention_ext_kv_noalloc",
                 "extkv_clear_status", "extkv_read_status", "extkv_set_algo"):
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return EXTKV_F32
    if t.dtype == torch.bfloat16:
        return EXTKV_BF16
    raise TypeError(f"unsupported element type {t.dtype}")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(code: int):
    if code != EXTKV_OK:
        raise ExtKVError(code, load().extkv_last_error().decode())


class PreparedCall:
    """One library call with its arguments marshalled once (pointers, sizes,
    the bias specification, the stream): calling it issues the same C call
    again, without the per-call checks and conversions of the Python layer.
    For a step repeated over the same buffers; the tensors it was prepared
    with must stay alive and in place, and their contents may change between
    calls."""

    __slots__ = ("_fn", "_args", "_keep")

    def __init__(self, fn, args, keep=()):
        self._fn = fn
        # ctypes instances of the declared argument types: the call converts nothing
        self._args = tuple(a if a is None or isinstance(a, ctypes._SimpleCData) or type(a).__name__ == "CArgObject"
                           else t(a) for a, t in zip(args, fn.argtypes))
        self._keep = keep  # the objects the pointers refer to (bias specification, workspace, tensors)

    def __call__(self):
        code = self._fn(*self._args)
        if code != EXTKV_OK:
            raise ExtKVError(code, load().extkv_last_error().decode())


def _need(t, name, dims=None, dtype=None):
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


_recording = {}  # stream handle of each open StepRecorder -> the workspaces its step needs


def _need_workspace(workspace, need, device, stream):
    """The caller's workspace, or one from the pool of the stream the call runs
    on (memory that is given back while the kernels run is then reused behind
    them).  One for a call that is being recorded stays with its step, which
    uses it again at every launch."""
    if workspace is None:
        if not need:
            return None
        handle = _stream(stream) or 0
        if handle == torch.cuda.current_stream().cuda_stream:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(handle)):
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
        if handle in _recording:
            _recording[handle].append(workspace)
        return workspace
    _need(workspace, "workspace")
    return workspace


@dataclass
class BiasSpec:
    """extkv_bias_spec: causal + sliding window + image spans + padding, with an
    optional dense extra term; tensors live on the device."""
    causal: bool = True
    window: int = 0
    span_offsets: Optional[torch.Tensor] = None  # (B+1,) int64
    spans: Optional[torch.Tensor] = None         # (n,2) int64
    extra: Optional[torch.Tensor] = None         # (B,1,S_q,max_seq)
    q_start: Optional[torch.Tensor] = None       # (B,) int64

    def _c(self) -> _BiasSpec:
        for t, n in ((self.span_offsets, "span_offsets"), (self.spans, "spans"),
                     (self.q_start, "q_start")):
            _need(t, n, dtype=torch.int64)
        _need(self.extra, "extra", dims=4)
        return _BiasSpec(int(bool(self.causal)), int(self.window), _p(self.span_offsets),
                         _p(self.spans), _p(self.extra), _p(self.q_start))


def ext_kv_scatter(k_cache, v_cache, k_new, v_new, write_idx, status=None, stream=None):
    """TensorScatter of (B,Hkv,S_new,D) rows into the (B,Hkv,max_seq,D) caches at write_idx."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (k_new, "k_new"), (v_new, "v_new")):
        _need(t, n, dims=4, dtype=k_cache.dtype)
    _need(write_idx, "write_idx", dims=1, dtype=torch.int64)
    B, Hkv, max_seq, D = k_cache.shape
    if v_cache.shape != k_cache.shape or k_new.shape != v_new.shape or k_new.shape[:2] != (B, Hkv) \
            or k_new.shape[3] != D:
        raise ValueError("inconsistent cache / update shapes")
    _check(load().ext_kv_scatter(_p(k_cache), _p(v_cache), _p(k_new), _p(v_new), _p(write_idx), B,
                                 Hkv, k_new.shape[2], max_seq, D, _dt(k_cache), _p(status),
                                 _stream(stream)))


def _marshal_bias(bias, spec: BiasSpec, nonpad, status, stream):
    _need(bias, "bias", dims=4)
    _need(nonpad, "nonpad", dims=1, dtype=torch.int64)
    B, one, S_q, max_seq = bias.shape
    if one != 1:
        raise ValueError("bias must be (B,1,S_q,max_seq)")
    c = spec._c()
    lib = load()
    return lib.build_static_cache_bias, (_p(bias), ctypes.byref(c), _p(nonpad), B, S_q, max_seq, _dt(bias),
                                         _p(status), _stream(stream)), (c, bias, nonpad, status)


def build_static_cache_bias(bias, spec: BiasSpec, nonpad, status=None, stream=None):
    """Materialise the (B,1,S_q,max_seq) bias of ``spec`` into ``bias``."""
    fn, args, _ = _marshal_bias(bias, spec, nonpad, status, stream)
    _check(fn(*args))


def prepare_build_static_cache_bias(bias, spec: BiasSpec, nonpad, status=None, stream=None) -> PreparedCall:
    """build_static_cache_bias with its arguments marshalled once (PreparedCall)."""
    return PreparedCall(*_marshal_bias(bias, spec, nonpad, status, stream))


def attention_ext_kv_workspace_size(B, Hq, Hkv, S_q, max_seq, D, dtype, Dv=None) -> int:
    """Bytes of device workspace attention_ext_kv needs (queries the current device);
    ``Dv``: the value head size when it differs from D."""
    dt = EXTKV_F32 if dtype == torch.float32 else EXTKV_BF16
    if Dv is None or Dv == D:
        return int(load().attention_ext_kv_workspace_size(B, Hq, Hkv, S_q, max_seq, D, dt))
    return int(load().attention_ext_kv_workspace_size_dv(B, Hq, Hkv, S_q, max_seq, D, Dv, dt))


def new_workspace(q: torch.Tensor, k_cache: torch.Tensor, v_cache: Optional[torch.Tensor] = None
                  ) -> Optional[torch.Tensor]:
    """A workspace sized for attention over these q / cache shapes (None if none is needed)."""
    B, Hq, S_q, D = q.shape
    Dv = D if v_cache is None else v_cache.shape[3]
    n = attention_ext_kv_workspace_size(B, Hq, k_cache.shape[1], S_q, k_cache.shape[2], D, q.dtype, Dv)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def _marshal_attention(y, q, k_cache, v_cache, nonpad, scale, bias, fused, workspace, status, stream, softcap):
    for t, n in ((y, "y"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, dims=4, dtype=q.dtype)
    _need(bias, "bias", dims=4, dtype=q.dtype)
    _need(nonpad, "nonpad", dims=1, dtype=torch.int64)
    B, Hq, S_q, D = q.shape
    Hkv, max_seq = k_cache.shape[1], k_cache.shape[2]
    Dv = v_cache.shape[3]
    if y.shape != (B, Hq, S_q, Dv) or v_cache.shape[:3] != k_cache.shape[:3] or k_cache.shape[0] != B or \
            k_cache.shape[3] != D:
        raise ValueError("inconsistent q / y / cache shapes")
    c = None if fused is None else fused._c()
    if workspace is None:
        need = attention_ext_kv_workspace_size(B, Hq, Hkv, S_q, max_seq, D, q.dtype, Dv)
        workspace = _need_workspace(None, need, q.device, stream)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    lib = load()
    keep = (c, workspace, y, q, k_cache, v_cache, bias, nonpad, status)
    args = (_p(y), _p(q), _p(k_cache), _p(v_cache), _p(bias), None if c is None else ctypes.byref(c), _p(nonpad),
            float(scale))
    if Dv != D:
        return lib.attention_ext_kv_dv, (*args, float(softcap), B, Hq, Hkv, S_q, max_seq, D, Dv, _dt(q),
                                         _p(workspace), ws, _p(status), _stream(stream)), keep
    tail = (B, Hq, Hkv, S_q, max_seq, D, _dt(q), _p(workspace), ws, _p(status), _stream(stream))
    if softcap:
        return lib.attention_ext_kv_softcap, (*args, float(softcap), *tail), keep
    return lib.attention_ext_kv, (*args, *tail), keep


def attention_ext_kv(y, q, k_cache, v_cache, nonpad, scale, bias=None, fused: Optional[BiasSpec] = None,
                     workspace=None, status=None, stream=None, softcap: float = 0.0):
    """Y = softmax(cap(scale*QK^T) + bias)V over the external cache; writes ``y`` (B,Hq,S_q,Dv).
    ``softcap`` > 0 caps the scaled scores to softcap*tanh(x/softcap) before the
    bias (attention_ext_kv_softcap); 0 is plain attention_ext_kv.  A v_cache
    whose head size Dv differs from q's and k_cache's Dk goes through
    attention_ext_kv_dv.

    ``workspace`` (uint8 device tensor of attention_ext_kv_workspace_size bytes)
    is allocated here when not given."""
    fn, args, _ = _marshal_attention(y, q, k_cache, v_cache, nonpad, scale, bias, fused, workspace, status,
                                     stream, softcap)
    _check(fn(*args))


def prepare_attention_ext_kv(y, q, k_cache, v_cache, nonpad, scale, bias=None, fused: Optional[BiasSpec] = None,
                             workspace=None, status=None, stream=None, softcap: float = 0.0) -> PreparedCall:
    """attention_ext_kv with its arguments marshalled once (PreparedCall); the
    workspace, when not given, is allocated here and kept by the call."""
    return PreparedCall(*_marshal_attention(y, q, k_cache, v_cache, nonpad, scale, bias, fused, workspace,
                                            status, stream, softcap))


def build_bias_from_bool_mask(bias, mask, stream=None):
    """Writes the additive bias of a boolean (B,1,S_q,max_seq) mask into ``bias``
    (same shape, float32 or bfloat16): 0 where the mask is true, the element
    type's lowest finite value where it is false."""
    _need(bias, "bias", dims=4)
    _need(mask, "mask", dims=4, dtype=torch.bool)
    if mask.shape != bias.shape or bias.shape[1] != 1:
        raise ValueError("mask and bias must both be (B,1,S_q,max_seq)")
    B, _, S_q, max_seq = bias.shape
    _check(load().build_bias_from_bool_mask(_p(bias), _p(mask), B, S_q, max_seq, _dt(bias), _stream(stream)))


def _marshal_attention_scatter(y, q, k_cache, v_cache, k_new, v_new, write_idx, nonpad, scale, bias, fused,
                               workspace, status, stream):
    for t, n in ((y, "y"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (k_new, "k_new"),
                 (v_new, "v_new")):
        _need(t, n, dims=4, dtype=q.dtype)
    _need(bias, "bias", dims=4, dtype=q.dtype)
    _need(nonpad, "nonpad", dims=1, dtype=torch.int64)
    _need(write_idx, "write_idx", dims=1, dtype=torch.int64)
    B, Hq, S_q, D = q.shape
    Hkv, max_seq = k_cache.shape[1], k_cache.shape[2]
    S_new = k_new.shape[2]
    if y.shape != q.shape or v_cache.shape != k_cache.shape or k_cache.shape[0] != B or \
            k_cache.shape[3] != D or k_new.shape != v_new.shape or k_new.shape[:2] != (B, Hkv) or \
            k_new.shape[3] != D or write_idx.shape[0] != B:
        raise ValueError("inconsistent q / y / cache / new-row shapes")
    c = None if fused is None else fused._c()
    if workspace is None:
        need = load().attention_ext_kv_workspace_size(B, Hq, Hkv, S_q, max_seq, D, _dt(q))
        workspace = _need_workspace(None, need, q.device, stream)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    keep = (c, workspace, y, q, k_cache, v_cache, k_new, v_new, write_idx, bias, nonpad, status)
    return load().attention_ext_kv_scatter, (_p(y), _p(q), _p(k_cache), _p(v_cache), _p(k_new), _p(v_new),
                                             _p(write_idx), S_new, _p(bias),
                                             None if c is None else ctypes.byref(c), _p(nonpad), float(scale),
                                             B, Hq, Hkv, S_q, max_seq, D, _dt(q), _p(workspace), ws,
                                             _p(status), _stream(stream)), keep


def attention_ext_kv_scatter(y, q, k_cache, v_cache, k_new, v_new, write_idx, nonpad, scale, bias=None,
                             fused: Optional[BiasSpec] = None, workspace=None, status=None, stream=None):
    """ext_kv_scatter of (k_new, v_new) at write_idx, then attention_ext_kv over
    the updated caches, in one call (fused into the decode kernel where it runs)."""
    fn, args, _ = _marshal_attention_scatter(y, q, k_cache, v_cache, k_new, v_new, write_idx, nonpad, scale,
                                             bias, fused, workspace, status, stream)
    _check(fn(*args))


def prepare_attention_ext_kv_scatter(y, q, k_cache, v_cache, k_new, v_new, write_idx, nonpad, scale, bias=None,
                                     fused: Optional[BiasSpec] = None, workspace=None, status=None,
                                     stream=None) -> PreparedCall:
    """attention_ext_kv_scatter with its arguments marshalled once (PreparedCall)."""
    return PreparedCall(*_marshal_attention_scatter(y, q, k_cache, v_cache, k_new, v_new, write_idx, nonpad,
                                                    scale, bias, fused, workspace, status, stream))


def attention_ext_kv_noalloc(y, q, k_cache, v_cache, nonpad, scale, bias=None,
                             fused: Optional[BiasSpec] = None, status=None, stream=None):
    """attention_ext_kv without a workspace, for callers that cannot allocate
    device memory (for instance an operator that is handed only its input and
    output buffers).  Decode shapes only; the scratch is a static 8 MiB array
    inside the library, shared by every call on the device, so calls that may
    overlap on the GPU must not use it concurrently."""
    for t, n in ((y, "y"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, dims=4, dtype=q.dtype)
    _need(bias, "bias", dims=4, dtype=q.dtype)
    _need(nonpad, "nonpad", dims=1, dtype=torch.int64)
    B, Hq, S_q, D = q.shape
    Hkv, max_seq = k_cache.shape[1], k_cache.shape[2]
    if y.shape != q.shape or v_cache.shape != k_cache.shape or k_cache.shape[0] != B or \
            k_cache.shape[3] != D:
        raise ValueError("inconsistent q / y / cache shapes")
    c = None if fused is None else fused._c()
    _check(load().attention_ext_kv_noalloc(_p(y), _p(q), _p(k_cache), _p(v_cache), _p(bias),
                                           None if c is None else ctypes.byref(c), _p(nonpad),
                                           float(scale), B, Hq, Hkv, S_q, max_seq, D, _dt(q),
                                           _p(status), _stream(stream)))


# ---- packed rows and a cache in pages ------------------------------------------------


@dataclass
class RotarySpec:
    """extkv_rotary: rotary positions with one to four axes.  ``positions``
    (axes, rows) int64 -- (axes, B, S) for rotary_multi_axis -- and ``inv_freq``
    (rotary_dim/2,) float32 live on the device; pair i is turned by
    positions[axis of i] * inv_freq[i], ``sections`` giving the pairs of each
    axis in turn.  Pairs are elements (i, i + rotary_dim/2), or (2i, 2i+1) when
    ``interleaved``."""
    positions: torch.Tensor
    inv_freq: torch.Tensor
    sections: Sequence[int]
    interleaved: bool = False

    def _c(self, shape) -> _Rotary:
        _need(self.inv_freq, "inv_freq", dims=1, dtype=torch.float32)
        _need(self.positions, "positions", dtype=torch.int64)
        n = len(self.sections)
        if not 1 <= n <= 4:
            raise ValueError("sections must name one to four axes")
        if tuple(self.positions.shape) != (n, *shape):
            raise ValueError(f"positions must be {(n, *shape)}, got {tuple(self.positions.shape)}")
        if sum(self.sections) != self.inv_freq.shape[0]:
            raise ValueError("sections must sum to the length of inv_freq (rotary_dim/2)")
        return _Rotary(n, (ctypes.c_int32 * 4)(*[int(x) for x in self.sections]), 2 * self.inv_freq.shape[0],
                       int(bool(self.interleaved)), _p(self.positions), _p(self.inv_freq))


def _on_current_device(**tensors):
    """Every tensor given is on the current CUDA device, where the call launches."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _need_rows(t, name, shape, dtype) -> int:
    """(rows, H, D) with dense (H, D) rows; returns the elements between rows."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    rows, H, D = shape
    if t.numel() and ((D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D)):
        raise ValueError(f"the heads of {name} must be dense within a row")
    return t.stride(0) if rows > 1 else H * D


def _window(window) -> int:
    """A window of 2^31 keys or more masks nothing that one of 2^31 - 1 does not."""
    return max(0, min(int(window), 2 ** 31 - 1))


def _need_status(status):
    _need(status, "status", dtype=torch.int32)
    if status is not None and status.numel() < 4:
        raise ValueError("status must hold 16 bytes")


def _marshal_rotary(q_out, k_out, q, k, rotary: RotarySpec, stream):
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    for t, o, n in ((q, q_out, "q"), (k, k_out, "k")):
        if (t is None) != (o is None):
            raise ValueError(f"{n} and {n}_out must be given together")
        _need(t, n, dims=4, dtype=first.dtype)
        _need(o, n + "_out", dims=4, dtype=first.dtype)
        if t is not None and (o.shape != t.shape or t.shape[0] != first.shape[0] or t.shape[2:] != first.shape[2:]):
            raise ValueError("inconsistent q / k shapes")
    B, _, S, D = first.shape
    dt = _dt(first)
    c = rotary._c((B, S))
    _on_current_device(q=q, q_out=q_out, k=k, k_out=k_out, positions=rotary.positions, inv_freq=rotary.inv_freq)
    return load().rotary_multi_axis, (_p(q_out), _p(k_out), _p(q), _p(k), ctypes.byref(c), B,
                                      1 if q is None else q.shape[1], 1 if k is None else k.shape[1], S, D, dt,
                                      _stream(stream)), (c, q_out, k_out, q, k, rotary)


def rotary_multi_axis(q_out, k_out, q, k, rotary: RotarySpec, stream=None):
    """Rotates q (B,Hq,S,D) into ``q_out`` and k (B,Hkv,S,D) into ``k_out`` by the
    angles of ``rotary`` (positions (axes,B,S)); either pair may be None, and an
    output may be its input."""
    fn, args, _ = _marshal_rotary(q_out, k_out, q, k, rotary, stream)
    _check(fn(*args))


def prepare_rotary_multi_axis(q_out, k_out, q, k, rotary: RotarySpec, stream=None) -> PreparedCall:
    """rotary_multi_axis with its arguments marshalled once (PreparedCall)."""
    return PreparedCall(*_marshal_rotary(q_out, k_out, q, k, rotary, stream))


def _need_pages(k_pages, v_pages, page_table, B, dtype):
    for t, n in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        _need(t, n, dims=4, dtype=dtype)
    if v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")
    _need(page_table, "page_table", dims=2, dtype=torch.int64)
    if page_table.shape[0] != B:
        raise ValueError(f"page_table must have {B} rows, got {page_table.shape[0]}")


def _marshal_append(k_pages, v_pages, k_new, v_new, page_table, write_idx, cu_seqlens, rotary, q_out, q, status,
                    stream):
    dtype = k_pages.dtype
    _need(write_idx, "write_idx", dims=1, dtype=torch.int64)
    B = write_idx.shape[0]
    _need_pages(k_pages, v_pages, page_table, B, dtype)
    num_pages, Hkv, page_size, D = k_pages.shape
    if k_new.dim() != 3:
        raise ValueError(f"k_new must have 3 dims, got {tuple(k_new.shape)}")
    T = k_new.shape[0]
    ks = _need_rows(k_new, "k_new", (T, Hkv, D), dtype)
    vs = _need_rows(v_new, "v_new", (T, Hkv, D), dtype)
    _need(cu_seqlens, "cu_seqlens", dims=1, dtype=torch.int64)
    if cu_seqlens is not None and cu_seqlens.shape[0] != B + 1:
        raise ValueError(f"cu_seqlens must have {B + 1} entries, got {cu_seqlens.shape[0]}")
    if cu_seqlens is None and T != B:
        raise ValueError(f"without cu_seqlens there is one row per sequence: {T} rows for {B} sequences")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out must be given together")
    qs, Hq = 0, 1
    if q is not None:
        if rotary is None:
            raise ValueError("q is rotated; it needs rotary")
        if q.dim() != 3:
            raise ValueError(f"q must have 3 dims, got {tuple(q.shape)}")
        Hq = q.shape[1]
        qs = _need_rows(q, "q", (T, Hq, D), dtype)
        _need(q_out, "q_out", dims=3, dtype=dtype)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    _need_status(status)
    dt = _dt(k_pages)
    c = None if rotary is None else rotary._c((T,))
    _on_current_device(k_pages=k_pages, v_pages=v_pages, k_new=k_new, v_new=v_new, page_table=page_table,
                       write_idx=write_idx, cu_seqlens=cu_seqlens, q=q, q_out=q_out, status=status,
                       positions=None if rotary is None else rotary.positions,
                       inv_freq=None if rotary is None else rotary.inv_freq)
    return load().paged_kv_append, (_p(k_pages), _p(v_pages), _p(k_new), _p(v_new), _p(page_table), _p(write_idx),
                                    _p(cu_seqlens), _p(q_out), _p(q), None if c is None else ctypes.byref(c), T, B, Hq,
                                    Hkv, D, num_pages, page_size, page_table.shape[1], qs, ks, vs, dt, _p(status),
                                    _stream(stream)), \
        (c, k_pages, v_pages, k_new, v_new, page_table, write_idx, cu_seqlens, rotary, q_out, q, status)


def paged_kv_append(k_pages, v_pages, k_new, v_new, page_table, write_idx, cu_seqlens=None,
                    rotary: Optional[RotarySpec] = None, q_out=None, q=None, status=None, stream=None):
    """Writes packed rows k_new, v_new (T,Hkv,D) into the pages
    (num_pages,Hkv,page_size,D) at slots write_idx[b].. of each sequence
    (cu_seqlens None: one row per sequence).  With ``rotary`` (positions
    (axes,T)) the K rows are rotated on the way, and q (T,Hq,D) into ``q_out``
    when given.  k_new, v_new and q may have any row stride that is a multiple
    of 16 bytes."""
    fn, args, _ = _marshal_append(k_pages, v_pages, k_new, v_new, page_table, write_idx, cu_seqlens, rotary, q_out, q,
                                  status, stream)
    _check(fn(*args))


def prepare_paged_kv_append(k_pages, v_pages, k_new, v_new, page_table, write_idx, cu_seqlens=None,
                            rotary: Optional[RotarySpec] = None, q_out=None, q=None, status=None,
                            stream=None) -> PreparedCall:
    """paged_kv_append with its arguments marshalled once (PreparedCall)."""
    return PreparedCall(*_marshal_append(k_pages, v_pages, k_new, v_new, page_table, write_idx, cu_seqlens, rotary,
                                         q_out, q, status, stream))


def attention_paged_decode_workspace_size(B, Hq, Hkv, D, dtype) -> int:
    """Bytes of device workspace attention_paged_decode needs (queries the current device)."""
    dt = EXTKV_F32 if dtype == torch.float32 else EXTKV_BF16
    return int(load().attention_paged_decode_workspace_size(B, Hq, Hkv, D, dt))


def _ws_bytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def _marshal_paged_decode(y, q, k_pages, v_pages, page_table, nonpad, scale, window, workspace, status, stream):
    if q.dim() != 3:
        raise ValueError(f"q must have 3 dims, got {tuple(q.shape)}")
    B, Hq, D = q.shape
    qs = _need_rows(q, "q", (B, Hq, D), q.dtype)
    _need(y, "y", dims=3, dtype=q.dtype)
    _need_pages(k_pages, v_pages, page_table, B, q.dtype)
    _need(nonpad, "nonpad", dims=1, dtype=torch.int64)
    num_pages, Hkv, page_size, Dk = k_pages.shape
    if y.shape != q.shape or Dk != D or nonpad.shape[0] != B:
        raise ValueError("inconsistent q / y / pages / nonpad shapes")
    _need_status(status)
    dt = _dt(q)
    _on_current_device(y=y, q=q, k_pages=k_pages, v_pages=v_pages, page_table=page_table, nonpad=nonpad,
                       workspace=workspace, status=status)
    workspace = _need_workspace(workspace, attention_paged_decode_workspace_size(B, Hq, Hkv, D, q.dtype), q.device,
                                stream)
    return load().attention_paged_decode, (_p(y), _p(q), _p(k_pages), _p(v_pages), _p(page_table), _p(nonpad),
                                           float(scale), _window(window), B, Hq, Hkv, D, num_pages, page_size,
                                           page_table.shape[1], qs, dt, _p(workspace), _ws_bytes(workspace),
                                           _p(status), _stream(stream)), \
        (workspace, y, q, k_pages, v_pages, page_table, nonpad, status)


def attention_paged_decode(y, q, k_pages, v_pages, page_table, nonpad, scale, window: int = 0, workspace=None,
                           status=None, stream=None):
    """Attention of one new token per sequence, q (B,Hq,D), over its first
    ``nonpad[b]`` slots (the last ``window`` of them when window > 0) in the
    pages (num_pages,Hkv,page_size,D); writes ``y`` (B,Hq,D).  The workspace is
    allocated here when not given (and stays with the step where the call is
    recorded into one)."""
    fn, args, _ = _marshal_paged_decode(y, q, k_pages, v_pages, page_table, nonpad, scale, window, workspace, status,
                                        stream)
    _check(fn(*args))


def prepare_attention_paged_decode(y, q, k_pages, v_pages, page_table, nonpad, scale, window: int = 0,
                                   workspace=None, status=None, stream=None) -> PreparedCall:
    """attention_paged_decode with its arguments marshalled once (PreparedCall)."""
    return PreparedCall(*_marshal_paged_decode(y, q, k_pages, v_pages, page_table, nonpad, scale, window, workspace,
                                               status, stream))


def attention_packed_prefill_workspace_size(T, B, Hq, Hkv, D, dtype) -> int:
    """Bytes of device workspace attention_packed_prefill needs (queries the current device)."""
    dt = EXTKV_F32 if dtype == torch.float32 else EXTKV_BF16
    return int(load().attention_packed_prefill_workspace_size(T, B, Hq, Hkv, D, dt))


def _marshal_packed_prefill(y, q, k, v, cu_seqlens, scale, causal, window, workspace, status, stream):
    for t, n in ((q, "q"), (k, "k")):
        if t.dim() != 3:
            raise ValueError(f"{n} must have 3 dims, got {tuple(t.shape)}")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    qs = _need_rows(q, "q", (T, Hq, D), q.dtype)
    ks = _need_rows(k, "k", (T, Hkv, D), q.dtype)
    vs = _need_rows(v, "v", (T, Hkv, D), q.dtype)
    _need(y, "y", dims=3, dtype=q.dtype)
    if y.shape != q.shape:
        raise ValueError("y must have q's shape")
    _need(cu_seqlens, "cu_seqlens", dims=1, dtype=torch.int64)
    if cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    B = cu_seqlens.shape[0] - 1
    _need_status(status)
    dt = _dt(q)
    _on_current_device(y=y, q=q, k=k, v=v, cu_seqlens=cu_seqlens, workspace=workspace, status=status)
    workspace = _need_workspace(workspace, attention_packed_prefill_workspace_size(T, B, Hq, Hkv, D, q.dtype),
                                q.device, stream)
    return load().attention_packed_prefill, (_p(y), _p(q), _p(k), _p(v), _p(cu_seqlens), float(scale),
                                             int(bool(causal)), _window(window), T, B, Hq, Hkv, D, qs, ks, vs, dt,
                                             _p(workspace), _ws_bytes(workspace), _p(status), _stream(stream)), \
        (workspace, y, q, k, v, cu_seqlens, status)


def attention_packed_prefill(y, q, k, v, cu_seqlens, scale, causal: bool = True, window: int = 0, workspace=None,
                             status=None, stream=None):
    """Attention over whole prompts packed one after another: q (T,Hq,D),
    k, v (T,Hkv,D), sequence b in rows cu_seqlens[b]..cu_seqlens[b+1]-1; writes
    the sequences' rows of ``y`` (T,Hq,D).  q, k and v may have any row stride
    that is a multiple of 16 bytes.  The workspace is allocated here when not
    given (and stays with the step where the call is recorded into one)."""
    fn, args, _ = _marshal_packed_prefill(y, q, k, v, cu_seqlens, scale, causal, window, workspace, status, stream)
    _check(fn(*args))


def prepare_attention_packed_prefill(y, q, k, v, cu_seqlens, scale, causal: bool = True, window: int = 0,
                                     workspace=None, status=None, stream=None) -> PreparedCall:
    """attention_packed_prefill with its arguments marshalled once (PreparedCall)."""
    return PreparedCall(*_marshal_packed_prefill(y, q, k, v, cu_seqlens, scale, causal, window, workspace, status,
                                                 stream))


def new_status(device="cuda") -> torch.Tensor:
    """A zeroed 16-byte device status word."""
    return torch.zeros(4, dtype=torch.int32, device=device)


def extkv_clear_status(status, stream=None):
    _check(load().extkv_clear_status(_p(status), _stream(stream)))


def extkv_read_status(status, stream=None) -> int:
    """Synchronises; returns EXTKV_OK or EXTKV_ERR_DEVICE (message in extkv_last_error)."""
    code = load().extkv_read_status(_p(status), _stream(stream))
    if code not in (EXTKV_OK, EXTKV_ERR_DEVICE):
        _check(code)
    return code


def extkv_last_error() -> str:
    return load().extkv_last_error().decode()


def extkv_last_kernel() -> str:
    return load().extkv_last_kernel().decode()


def extkv_last_launches() -> int:
    """Kernels the calling thread's last attention_ext_kv launched."""
    return int(load().extkv_last_launches())


def extkv_set_algo(algo: int) -> int:
    prev = load().extkv_set_algo(int(algo))
    if prev < 0:
        _check(prev)
    return prev


def extkv_set_wait_polls(polls: int) -> int:
    """Poll limit of the kernels' pipeline waits for this thread (0: give up
    at once; negative: the kernels' own limit); returns the previous setting.
    For failure-detection tests."""
    return int(load().extkv_set_wait_polls(int(polls)))


class wait_polls:
    """Context manager setting the pipeline-wait poll limit for the calling thread."""

    def __init__(self, polls: int):
        self.polls = polls

    def __enter__(self):
        self.prev = extkv_set_wait_polls(self.polls)
        return self

    def __exit__(self, *exc):
        extkv_set_wait_polls(self.prev)


class use_algo:
    """Context manager forcing one attention kernel for the calling thread."""

    def __init__(self, algo: int):
        self.algo = algo

    def __enter__(self):
        self.prev = extkv_set_algo(self.algo)
        return self

    def __exit__(self, *exc):
        extkv_set_algo(self.prev)


class RecordedStep:
    """A step recorded with StepRecorder: calling it starts every recorded
    library call again with one launch, on ``stream`` (a torch stream or a raw
    handle; default the current stream).  It keeps the workspaces that its calls
    allocated; the tensors they were given must stay alive and in place.  A step
    launched on a raw handle is kept until its launches have finished."""

    __slots__ = ("_h", "_workspaces", "_noted")

    def __init__(self, handle: int, workspaces=()):
        self._h = ctypes.c_void_p(handle)
        self._workspaces = list(workspaces)
        self._noted = set()  # streams behind whose launches freed workspaces are reused

    def __call__(self, stream=None):
        handle = _stream(stream)
        if self._workspaces and handle not in self._noted and not isinstance(stream, (int, torch.cuda.ExternalStream)):
            self._noted.add(handle)
            for w in self._workspaces:
                w.record_stream(torch.cuda.current_stream() if stream is None else stream)
        code = load().extkv_step_launch(self._h, handle)
        if code != EXTKV_OK:
            raise ExtKVError(code, load().extkv_last_error().decode())

    def __del__(self):
        if _lib is not None and self._h:
            _lib.extkv_step_free(self._h)
            self._h = ctypes.c_void_p()


class StepRecorder:
    """Records the library calls issued with ``stream=rec.stream`` inside the
    block into ``rec.step`` (extkv_step_begin / extkv_step_end).  Issue each
    call once before recording it, and call nothing that synchronises inside."""

    def __enter__(self):
        h = ctypes.c_void_p()
        _check(load().extkv_step_begin(ctypes.byref(h)))
        self.stream = h.value
        self.step = None
        _recording[self.stream] = []
        return self

    def __exit__(self, exc_type, exc, tb):
        out = ctypes.c_void_p()
        workspaces = _recording.pop(self.stream, ())
        code = load().extkv_step_end(ctypes.c_void_p(self.stream), ctypes.byref(out))
        if exc_type is not None:
            if out.value:
                load().extkv_step_free(out)
            return False
        _check(code)
        self.step = RecordedStep(out.value, workspaces)
        return False
