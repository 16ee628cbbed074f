"""NF4 weight-only linear layer for NVIDIA GB300 (sm_103a): thin Python binding of libnf4.so.

The library (``csrc/``, C ABI in ``include/nf4.h``) does all the work.  This module only marshals
torch tensors (device memory and streams) into the C calls of the same names and raises
``NF4Error`` on a non-OK status.  There is no CPU fallback: if ``libnf4.so`` has not been built
(``nf4_weight_only_gb300.build.build()``), every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import warnings
from typing import Optional

import torch

from . import build as _build

GROUP = 64
# (torch.cuda.current_stream() builds a stream object, about a microsecond)
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
LIB_PATH = _build.LIB_PATH

STATUS_NAMES = {0: "NF4_OK", 1: "NF4_ERR_NULL", 2: "NF4_ERR_SHAPE", 3: "NF4_ERR_ALIGN",
                4: "NF4_ERR_ALIAS", 5: "NF4_ERR_UNSUPPORTED_DEVICE", 6: "NF4_ERR_CUDA", 7: "NF4_ERR_MEMORY",
                8: "NF4_ERR_CAPTURE"}

# Every symbol include/nf4.h declares.
EXPORTED = ("nf4_quantize", "nf4_dequant", "nf4_linear", "nf4_linear_grouped", "nf4_embed",
            "nf4_kv_append", "nf4_kv_read", "nf4_attention_workspace_bytes", "nf4_attention_decode", "nf4_rope",
            "nf4_rmsnorm", "nf4_ring_create", "nf4_ring_run", "nf4_ring_destroy", "nf4_linear_host_noalloc",
            "nf4_check_device_error", "nf4_diag_bounded_wait", "nf4_diag_set_wait_limit", "nf4_status_str",
            "nf4_abi_version", "nf4_noalloc_slot_bytes", "nf4_last_cuda_error")


class HostLinear(ctypes.Structure):
    """nf4_host_linear: one linear of a streamed list (x, y on the device; codes, scales pinned host)."""
    _fields_ = [("x", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class NF4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}")


_lib: Optional[ctypes.CDLL] = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libnf4.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with nf4_weight_only_gb300.build.build() "
                           "(no CPU fallback exists)")
    lib = ctypes.CDLL(p)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.nf4_quantize.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.nf4_quantize.restype = ci
    lib.nf4_dequant.argtypes = [vp, vp, i64, i64, vp, vp]
    lib.nf4_dequant.restype = ci
    lib.nf4_linear.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    lib.nf4_linear.restype = ci
    lib.nf4_linear_grouped.argtypes = [vp, i64, i64, ci, vp, vp, vp, vp, vp]
    lib.nf4_linear_grouped.restype = ci
    lib.nf4_embed.argtypes = [vp, i64, vp, vp, i64, i64, vp, vp]
    lib.nf4_embed.restype = ci
    cf = ctypes.c_float
    lib.nf4_kv_append.argtypes = [vp, vp, vp, vp, i64, vp]
    lib.nf4_kv_append.restype = ci
    lib.nf4_kv_read.argtypes = [vp, vp, i64, vp, vp, vp]
    lib.nf4_kv_read.restype = ci
    lib.nf4_attention_workspace_bytes.argtypes = [vp, i64, i64]
    lib.nf4_attention_workspace_bytes.restype = i64
    lib.nf4_attention_decode.argtypes = [vp, vp, vp, i64, vp, i64, i64, cf, i64, vp, vp, i64, vp]
    lib.nf4_attention_decode.restype = ci
    lib.nf4_rope.argtypes = [vp, i64, vp, i64, i64, i64, vp, ci, vp, vp, i64, ci, cf, vp, vp, vp]
    lib.nf4_rope.restype = ci
    lib.nf4_rmsnorm.argtypes = [vp, vp, vp, i64, i64, cf, vp, vp, vp, vp, vp]
    lib.nf4_rmsnorm.restype = ci
    lib.nf4_ring_create.argtypes = [i64, ctypes.POINTER(ctypes.c_void_p)]
    lib.nf4_ring_create.restype = ci
    lib.nf4_ring_run.argtypes = [vp, vp, i64, vp]
    lib.nf4_ring_run.restype = ci
    lib.nf4_ring_destroy.argtypes = [vp]
    lib.nf4_ring_destroy.restype = ci
    lib.nf4_linear_host_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    lib.nf4_linear_host_noalloc.restype = ci
    lib.nf4_status_str.argtypes = [ci]
    lib.nf4_status_str.restype = ctypes.c_char_p
    lib.nf4_check_device_error.argtypes = [ctypes.POINTER(ctypes.c_int)]
    lib.nf4_check_device_error.restype = ci
    lib.nf4_diag_bounded_wait.argtypes = [i64, vp]
    lib.nf4_diag_bounded_wait.restype = ci
    lib.nf4_diag_set_wait_limit.argtypes = [i64, vp]
    lib.nf4_diag_set_wait_limit.restype = ci
    lib.nf4_noalloc_slot_bytes.argtypes = []
    lib.nf4_noalloc_slot_bytes.restype = i64
    lib.nf4_last_cuda_error.argtypes = []
    lib.nf4_last_cuda_error.restype = ctypes.c_char_p
    lib.nf4_abi_version.argtypes = []
    lib.nf4_abi_version.restype = ci
    if path is None:
        _lib = lib
    return lib


_calls = None


class _NoCalls:
    """In the compiled calls' place where they were not built: every call goes through ctypes."""
    append = read = attention = rope = rmsnorm = staticmethod(lambda *args: None)


def _load_calls(lib: ctypes.CDLL) -> None:
    """The compiled short way into `lib` for the calls of a decode loop (csrc/nf4_python.c)."""
    global _calls
    if not os.path.exists(_build.CALLS_PATH):
        warnings.warn(f"{_build.CALLS_PATH} was not built: cache, attention, rope and norm calls go through ctypes, "
                      "which takes some microseconds more of the host's time", RuntimeWarning, stacklevel=3)
        _calls = _NoCalls
        return
    loader = importlib.machinery.ExtensionFileLoader("nf4_calls", _build.CALLS_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("nf4_calls", loader))
    loader.exec_module(module)
    functions = (lib.nf4_kv_append, lib.nf4_kv_read, lib.nf4_attention_decode, lib.nf4_rope, lib.nf4_rmsnorm)
    module.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in functions), torch.bfloat16, torch.float8_e4m3fn,
                torch.float32, torch.int32, torch.int64, torch.uint8, _raw_stream, _current_device)
    _calls = module


def status_str(status: int) -> str:
    try:
        return load().nf4_status_str(status).decode()
    except RuntimeError:
        return STATUS_NAMES.get(status, f"status {status}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _check(status: int, what: str) -> None:
    if status != 0:
        if status == 6:  # NF4_ERR_CUDA: name the CUDA error behind it
            raise NF4Error(status, f"{what} [{load().nf4_last_cuda_error().decode()}]")
        raise NF4Error(status, what)


def nf4_quantize(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """w fp32 [N, K] -> codes uint8 [N, K/2], scales fp16 [N, K/64] (all CUDA tensors)."""
    n, k = w.shape
    _check(load().nf4_quantize(_ptr(w), n, k, _ptr(codes), _ptr(scales), _stream(stream)), "nf4_quantize")


def nf4_dequant(codes: torch.Tensor, scales: torch.Tensor, w_hat: torch.Tensor, stream=None) -> None:
    """codes [N, K/2], scales [N, K/64] -> w_hat bf16 [N, K]."""
    n, k = codes.shape[0], codes.shape[1] * 2
    _check(load().nf4_dequant(_ptr(codes), _ptr(scales), n, k, _ptr(w_hat), _stream(stream)), "nf4_dequant")


def nf4_linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor,
               stream=None) -> None:
    """y[M, N] = x[M, K] * w_hat^T (bf16 in, bf16 out)."""
    m, k = x.shape
    n = codes.shape[0]
    _check(load().nf4_linear(_ptr(x), _ptr(codes), _ptr(scales), _ptr(y), m, n, k, _stream(stream)),
           "nf4_linear")


def nf4_linear_grouped(x: torch.Tensor, codes, scales, ys, stream=None) -> None:
    """ys[i][M, N_i] = x[M, K] * w_hat_i^T for the lists codes, scales, ys (same length, <= 8)."""
    m, k = x.shape
    n = len(codes)
    if not (len(scales) == len(ys) == n):
        raise ValueError("codes, scales and ys must have the same length")
    arr = ctypes.c_void_p * n
    c_arr = arr(*[_ptr(c).value for c in codes])
    s_arr = arr(*[_ptr(s).value for s in scales])
    y_arr = arr(*[_ptr(y).value for y in ys])
    ns = (ctypes.c_int64 * n)(*[c.shape[0] for c in codes])
    _check(load().nf4_linear_grouped(_ptr(x), m, k, n, ctypes.cast(c_arr, ctypes.c_void_p),
                                     ctypes.cast(s_arr, ctypes.c_void_p), ctypes.cast(y_arr, ctypes.c_void_p),
                                     ctypes.cast(ns, ctypes.c_void_p), _stream(stream)), "nf4_linear_grouped")


def nf4_embed(ids: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """out[i] = w_hat[ids[i]] for int32 ids, codes [V, K/2], scales [V, K/64] -> out bf16 [n, K]."""
    v, k = codes.shape[0], codes.shape[1] * 2
    _check(load().nf4_embed(_ptr(ids), ids.numel(), _ptr(codes), _ptr(scales), v, k, _ptr(out), _stream(stream)),
           "nf4_embed")


def nf4_ring_create(slot_bytes: int) -> int:
    """A ring of two device slots of `slot_bytes` each (returns the opaque handle)."""
    h = ctypes.c_void_p(0)
    _check(load().nf4_ring_create(slot_bytes, ctypes.byref(h)), "nf4_ring_create")
    return h.value


def nf4_ring_run(ring: int, ops, stream=None) -> None:
    """Stream a list of linears (x, codes, scales, y) through the ring: codes [N, K/2] and scales
    [N, K/64] in pinned host memory, x [M, K] and y [M, N] on the device."""
    arr = (HostLinear * max(1, len(ops)))()
    for i, (x, codes, scales, y) in enumerate(ops):
        arr[i] = HostLinear(_ptr(x).value, _ptr(codes).value, _ptr(scales).value, _ptr(y).value,
                            x.shape[0], codes.shape[0], x.shape[1])
    _check(load().nf4_ring_run(ctypes.c_void_p(ring), ctypes.cast(arr, ctypes.c_void_p), len(ops), _stream(stream)),
           "nf4_ring_run")


def nf4_ring_destroy(ring: int) -> None:
    _check(load().nf4_ring_destroy(ctypes.c_void_p(ring)), "nf4_ring_destroy")


class Ring:
    """Two reusable device slots through which packed weights in pinned host memory are streamed."""

    def __init__(self, slot_bytes: int):
        self.handle = nf4_ring_create(slot_bytes)
        self.slot_bytes = slot_bytes

    @staticmethod
    def bytes_needed(n: int, k: int) -> int:
        return (n * k // 2 + 255) // 256 * 256 + n * (k // GROUP) * 2

    def run(self, ops, stream=None) -> None:
        nf4_ring_run(self.handle, ops, stream)

    def close(self) -> None:
        if self.handle:
            nf4_ring_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def noalloc_slot_bytes() -> int:
    """Size of nf4_linear_host_noalloc's static device array, as the built library reports it."""
    return int(load().nf4_noalloc_slot_bytes())


def nf4_linear_host_noalloc(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor,
                            stream=None) -> None:
    """y[M, N] = x[M, K] * w_hat^T with codes [N, K/2] and scales [N, K/64] in pinned host memory,
    staged through the library's static device buffer (no allocation; at most noalloc_slot_bytes())."""
    m, k = x.shape
    n = codes.shape[0]
    _check(load().nf4_linear_host_noalloc(_ptr(x), _ptr(codes), _ptr(scales), _ptr(y), m, n, k, _stream(stream)),
           "nf4_linear_host_noalloc")


def nf4_diag_bounded_wait(ns: int, stream=None) -> None:
    """Launch one thread whose bounded wait on a barrier nothing arrives on runs out after `ns`
    nanoseconds and records code 39 in the device error word (diagnostics)."""
    _check(load().nf4_diag_bounded_wait(int(ns), _stream(stream)), "nf4_diag_bounded_wait")


def nf4_diag_set_wait_limit(ns: int, stream=None) -> None:
    """Set the per-wait wall-clock limit of the kernels' pipeline waits (ns = 0 restores 1 s)."""
    _check(load().nf4_diag_set_wait_limit(int(ns), _stream(stream)), "nf4_diag_set_wait_limit")


def nf4_check_device_error() -> int:
    """Read and clear the device error word (0 = no pipeline wait timed out).  Synchronizes."""
    code = ctypes.c_int(0)
    _check(load().nf4_check_device_error(ctypes.byref(code)), "nf4_check_device_error")
    return code.value


# ---------------------------------------------------------------------------------------------
# Operators around the linears of a decoder layer
# ---------------------------------------------------------------------------------------------
KV_FORMATS = {"bf16": 0, "fp8": 1, "nf4": 2}


class _KvCacheStruct(ctypes.Structure):
    """nf4_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


def _ready():
    """The compiled calls.  Each returns a status, or None for tensors that it does not take: the wrappers then go
    through their own checks, which say what is wrong, and through ctypes."""
    if _calls is None:
        _load_calls(load())
    return _calls


def _expect(t: torch.Tensor, name: str, dtype, shape) -> int:
    """The address of a contiguous CUDA tensor of exactly this type and shape (or ValueError)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: want a tensor, got {type(t).__name__}")
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    raise ValueError(f"{name}: want a CUDA tensor")


def _current(stream) -> int:
    """The raw handle of `stream`, or of the current device's current stream."""
    if stream is None:
        return _raw_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream):
    """Where results are allocated: on the stream that computes them.  (torch may hand out memory that the current
    stream still uses.)"""
    if stream is None:
        return contextlib.nullcontext()
    if hasattr(stream, "cuda_stream"):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream())


class KVCache:
    """A paged key-value cache over the caller's tensors (include/nf4.h, nf4_kv_cache).

    format "bf16": k, v bf16 [pages, kv_heads, page_size, head_dim]; no scales.
    format "fp8":  k, v float8_e4m3fn of that shape; scales fp32 [pages, kv_heads, page_size].
    format "nf4":  k, v uint8 [pages, kv_heads, page_size, head_dim/2]; scales fp16 [..., head_dim/64].
    """

    def __init__(self, format: str, k: torch.Tensor, v: torch.Tensor, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None):
        if format not in KV_FORMATS:
            raise ValueError(f"format {format!r}: want one of {sorted(KV_FORMATS)}")
        if k.dim() != 4:
            raise ValueError("k: want [pages, kv_heads, page_size, head_dim]")
        pages, kv_heads, page_size, width = k.shape
        head_dim = 2 * width if format == "nf4" else width
        dtype = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "nf4": torch.uint8}[format]
        places = (pages, kv_heads, page_size)
        pk, pv = _expect(k, "k", dtype, k.shape), _expect(v, "v", dtype, k.shape)
        pks = pvs = 0
        if format == "bf16":
            if k_scales is not None or v_scales is not None:
                raise ValueError("a bf16 cache has no scales")
        else:
            if k_scales is None or v_scales is None:
                raise ValueError(f"a cache in {format} needs k_scales and v_scales")
            sdtype, sshape = ((torch.float32, places) if format == "fp8" else
                              (torch.float16, (*places, head_dim // GROUP)))
            pks, pvs = _expect(k_scales, "k_scales", sdtype, sshape), _expect(v_scales, "v_scales", sdtype, sshape)
        self.format, self.pages, self.kv_heads = format, pages, kv_heads
        self.page_size, self.head_dim = page_size, head_dim
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.device = k.device
        self._c = _KvCacheStruct(pk, pv, pks, pvs, pages, kv_heads, page_size, head_dim, KV_FORMATS[format])
        self._address = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, format: str, pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> "KVCache":
        """A cache with its own tensors, zeroed."""
        places = (pages, kv_heads, page_size)

        def zeros(width, dtype):
            return torch.zeros((*places, width), dtype=dtype, device=device)

        if format == "bf16":
            return cls(format, zeros(head_dim, torch.bfloat16), zeros(head_dim, torch.bfloat16))
        if format == "fp8":
            side = [zeros(head_dim, torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)]
            return cls(format, *side, *(torch.zeros(places, dtype=torch.float32, device=device) for _ in range(2)))
        if format == "nf4":
            return cls(format, zeros(head_dim // 2, torch.uint8), zeros(head_dim // 2, torch.uint8),
                       zeros(head_dim // GROUP, torch.float16), zeros(head_dim // GROUP, torch.float16))
        raise ValueError(f"format {format!r}: want one of {sorted(KV_FORMATS)}")


def nf4_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Write k, v bf16 [T, kv_heads, head_dim] at int64 slots [T] (page * page_size + offset; < 0: skip)."""
    status = _ready().append(cache._address, cache.kv_heads, cache.head_dim, k, v, slots, stream)
    if status is not None:
        return _check(status, "nf4_kv_append")
    t = slots.shape[0]
    shape = (t, cache.kv_heads, cache.head_dim)
    _check(load().nf4_kv_append(cache._address, _expect(k, "k", torch.bfloat16, shape),
                                _expect(v, "v", torch.bfloat16, shape), _expect(slots, "slots", torch.int64, (t,)), t,
                                _current(stream)), "nf4_kv_append")


def nf4_kv_read(cache: KVCache, slots: torch.Tensor, k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                stream=None) -> None:
    """Read int64 slots [T] back into k and / or v bf16 [T, kv_heads, head_dim]."""
    status = _ready().read(cache._address, cache.kv_heads, cache.head_dim, slots, k, v, stream)
    if status is not None:
        return _check(status, "nf4_kv_read")
    t = slots.shape[0]
    shape = (t, cache.kv_heads, cache.head_dim)
    _check(load().nf4_kv_read(cache._address, _expect(slots, "slots", torch.int64, (t,)), t,
                              None if k is None else _expect(k, "k", torch.bfloat16, shape),
                              None if v is None else _expect(v, "v", torch.bfloat16, shape), _current(stream)),
           "nf4_kv_read")


def nf4_attention_workspace_bytes(cache: KVCache, batch: int, q_heads: int) -> int:
    n = load().nf4_attention_workspace_bytes(cache._address, batch, q_heads)
    if n < 0:
        raise NF4Error(2, "nf4_attention_workspace_bytes")
    return n


def attention_workspace(cache: KVCache, batch: int, q_heads: int, stream=None) -> torch.Tensor:
    """A workspace for nf4_attention_decode with this cache and these heads, allocated and zeroed on `stream`: calls
    on another stream wait for that first."""
    with _on(stream):
        return torch.zeros(nf4_attention_workspace_bytes(cache, batch, q_heads), dtype=torch.uint8, device=cache.device)


def nf4_attention_decode(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
                         out: torch.Tensor, workspace: torch.Tensor, scale: Optional[float] = None, window: int = 0,
                         stream=None) -> None:
    """out[b, h] = attention of q bf16 [B, q_heads, head_dim] over the cache's places of each sequence:
    page_table int32 [B, max_pages], lengths int32 [B]; scale defaults to head_dim ** -0.5."""
    status = _ready().attention(cache._address, cache.head_dim, q, page_table, lengths, out, workspace, scale, window,
                                stream)
    if status is not None:
        return _check(status, "nf4_attention_decode")
    shape, max_pages, size = q.shape, page_table.shape[-1], workspace.numel()
    b, q_heads, d = shape
    if d != cache.head_dim:
        raise ValueError(f"q: head_dim {d}, the cache has {cache.head_dim}")
    _check(load().nf4_attention_decode(
        cache._address, _expect(q, "q", torch.bfloat16, shape),
        _expect(page_table, "page_table", torch.int32, (b, max_pages)), max_pages,
        _expect(lengths, "lengths", torch.int32, (b,)), b, q_heads, d ** -0.5 if scale is None else scale, window,
        _expect(out, "out", torch.bfloat16, shape), _expect(workspace, "workspace", torch.uint8, (size,)), size,
        _current(stream)), "nf4_attention_decode")


def nf4_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor,
             q_out: Optional[torch.Tensor], k_out: Optional[torch.Tensor], sections=None, interleaved: bool = False,
             magnitude: float = 1.0, stream=None) -> None:
    """Rotary positions on q [T, q_heads, D] and k [T, k_heads, D] (bf16; either may be None; the outputs
    may be the inputs): positions int32 [axes, T], inv_freq fp32 [rotary_dim / 2], `sections` the pairs of
    each axis (default: one axis)."""
    status = _ready().rope(q, k, positions, inv_freq, q_out, k_out, sections, interleaved, magnitude, stream)
    if status is not None:
        return _check(status, "nf4_rope")
    one = q if q is not None else k
    if one is None:
        raise ValueError("q and k are both None")
    t, _, d = one.shape
    axes, pairs = positions.shape[0], inv_freq.shape[0]
    counts = _section_counts((pairs,) if sections is None else tuple(sections))
    if len(counts) != axes:
        raise ValueError(f"sections: want one count for each of the {axes} axes")
    bf16 = torch.bfloat16
    pq = hq = pqo = pk = hk = pko = 0
    if q is not None:
        hq = q.shape[1]
        pq, pqo = _expect(q, "q", bf16, (t, hq, d)), _expect(q_out, "q_out", bf16, (t, hq, d))
    if k is not None:
        hk = k.shape[1]
        pk, pko = _expect(k, "k", bf16, (t, hk, d)), _expect(k_out, "k_out", bf16, (t, hk, d))
    _check(load().nf4_rope(pq, hq, pk, hk, t, d, _expect(positions, "positions", torch.int32, (axes, t)), axes, counts,
                           _expect(inv_freq, "inv_freq", torch.float32, (pairs,)), 2 * pairs, int(interleaved),
                           magnitude, pqo, pko, _current(stream)), "nf4_rope")


@functools.lru_cache(maxsize=64)
def _section_counts(sections):
    """The counts as the host array nf4_rope reads."""
    return (ctypes.c_int32 * len(sections))(*sections)


def nf4_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                y8: Optional[torch.Tensor] = None, y8_scales: Optional[torch.Tensor] = None, stream=None) -> None:
    """Norm of x (+ residual) bf16 [T, H] into y bf16 and / or y8 float8_e4m3fn with y8_scales fp32 [T];
    residual_out receives the sum."""
    status = _ready().rmsnorm(x, weight, eps, residual, residual_out, y, y8, y8_scales, stream)
    if status is not None:
        return _check(status, "nf4_rmsnorm")
    bf16, shape = torch.bfloat16, x.shape
    t, h = shape
    _check(load().nf4_rmsnorm(_expect(x, "x", bf16, shape),
                              None if residual is None else _expect(residual, "residual", bf16, shape),
                              _expect(weight, "weight", bf16, (h,)), t, h, eps,
                              None if residual_out is None else _expect(residual_out, "residual_out", bf16, shape),
                              None if y is None else _expect(y, "y", bf16, shape),
                              None if y8 is None else _expect(y8, "y8", torch.float8_e4m3fn, shape),
                              None if y8_scales is None else _expect(y8_scales, "y8_scales", torch.float32, (t,)),
                              _current(stream)), "nf4_rmsnorm")


# Convenience wrappers that allocate the outputs with torch.
def kv_read(cache: KVCache, slots: torch.Tensor, stream=None):
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    with _on(stream):
        k, v = (torch.empty(shape, dtype=torch.bfloat16, device=slots.device) for _ in range(2))
    nf4_kv_read(cache, slots, k, v, stream)
    return k, v


def attention_decode(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
                     workspace: torch.Tensor, scale: Optional[float] = None, window: int = 0, stream=None):
    with _on(stream):
        out = torch.empty_like(q)
    nf4_attention_decode(cache, q, page_table, lengths, out, workspace, scale, window, stream)
    return out


def rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, sections=None,
         interleaved: bool = False, magnitude: float = 1.0, stream=None):
    with _on(stream):
        q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    nf4_rope(q, k, positions, inv_freq, q_out, k_out, sections, interleaved, magnitude, stream)
    return q_out, k_out


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None, stream=None):
    """y, or (y, x + residual) with a residual."""
    with _on(stream):
        y = torch.empty_like(x)
        r = None if residual is None else torch.empty_like(x)
    nf4_rmsnorm(x, weight, eps, residual=residual, residual_out=r, y=y, stream=stream)
    return y if residual is None else (y, r)


def quantize(w: torch.Tensor, stream=None):
    n, k = w.shape
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((n, k // GROUP), dtype=torch.float16, device=w.device)
    nf4_quantize(w, codes, scales, stream)
    return codes, scales


def dequant(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> torch.Tensor:
    w_hat = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.bfloat16, device=codes.device)
    nf4_dequant(codes, scales, w_hat, stream)
    return w_hat


def embed(ids: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> torch.Tensor:
    out = torch.empty((ids.numel(), codes.shape[1] * 2), dtype=torch.bfloat16, device=codes.device)
    nf4_embed(ids, codes, scales, out, stream)
    return out


def linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> torch.Tensor:
    y = torch.empty((x.shape[0], codes.shape[0]), dtype=torch.bfloat16, device=x.device)
    nf4_linear(x, codes, scales, y, stream)
    return y
