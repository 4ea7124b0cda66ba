"""The operators of include/pa_q4.h over torch CUDA tensors.

Every function checks its tensors, converts them to pointers and calls the C
ABI of the same name on the tensors' device and a stream of it (the current
one by default); all computation runs in the library's CUDA kernels.  Outputs
are written into tensors the caller passes, nothing is allocated, and no call
synchronises (the convenience call ``q4_decode`` does both).

A 4-bit cache is a uint8 tensor [num_pages, Hkv, 20 * D] (``new_q4_cache``).
It does not record its element type: read it with the dtype it was written
with.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import build as _build
from .binding import (PA_DTYPE_BF16, PA_DTYPE_F16, PA_DTYPE_F32, PA_OK, PAError, load,
                      new_workspace, pa_get_error)

PA_DEVERR_BAD_SLOT = 8
PA_DEVERR_NO_PAGES = 16
PAGE_SIZE = 16
_DTYPE = {torch.float16: PA_DTYPE_F16, torch.bfloat16: PA_DTYPE_BF16, torch.float32: PA_DTYPE_F32}
_TORCH = {v: k for k, v in _DTYPE.items()}

# The current stream's handle without a Stream object around it (1 us less).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class pa_q4_plan_t(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int),
        ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("num_pages", ctypes.c_int),
        ("max_pages_per_seq", ctypes.c_int),
        ("max_context_len", ctypes.c_int),
        ("window", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("num_sms", ctypes.c_int),
        ("heads_per_cta", ctypes.c_int),
        ("ctas_per_group", ctypes.c_int),
        ("ctas", ctypes.c_int),
        ("workspace_bytes", ctypes.c_size_t),
        ("ctrl_bytes", ctypes.c_int),
        ("test_stall_bytes", ctypes.c_int),
        ("cluster", ctypes.c_int),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


_bound = None
# The marshalling extension (csrc/pa_pyfast.cpp), once the library is loaded: it makes the usual
# call in a third of the host time, and returns None where it leaves a call to the code here.
_fast = None


def _load_fast(lib):
    path = _build.pyfast_path()  # (of these sources and this torch, or none)
    if _raw_stream is None or path is None or not os.path.exists(path):
        return None
    try:
        spec = importlib.util.spec_from_file_location("_pa_fast", path)
        fast = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(fast)
    except ImportError:  # built for another interpreter
        return None
    names = ("pa_q4_write", "pa_q4_read", "pa_q4_decode", "pa_extend_tables", "pa_rope_axes")
    fast.setup(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names),
               getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device), _raw_stream)
    return fast


def _lib():
    """The library with this module's signatures set."""
    global _bound, _fast
    if _bound is not None:
        return _bound
    lib = load()
    P, i, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
    plan = ctypes.POINTER(pa_q4_plan_t)
    lib.pa_q4_page_bytes.argtypes = [i]
    lib.pa_q4_page_bytes.restype = i
    lib.pa_q4_write.argtypes = [i] * 6 + [P, ll, P, ll, P, P, P, P]
    lib.pa_q4_write.restype = i
    lib.pa_q4_read.argtypes = [i] * 6 + [P, P, P, ll, P, ll, P, P]
    lib.pa_q4_read.restype = i
    lib.pa_q4_plan.argtypes = [i] * 11 + [plan]
    lib.pa_q4_plan.restype = i
    lib.pa_q4_decode.argtypes = [plan, P, P, P, P, ctypes.c_float, i, P, P, P, P]
    lib.pa_q4_decode.restype = i
    lib.pa_extend_tables.argtypes = [i] * 6 + [P] * 11
    lib.pa_extend_tables.restype = i
    lib.pa_rope_axes.argtypes = ([i] * 6 + [ctypes.POINTER(i), i, i, ctypes.c_float, i] +
                                 [P, ll, P, ll, P, P, ll, P, ll, P])
    lib.pa_rope_axes.restype = i
    _fast = _load_fast(lib)
    _bound = lib
    return lib


def _check(t, name, dtype, shape, dev):
    """Address of a contiguous CUDA tensor of this dtype, shape and device.

    (A small step's host time is these checks and the launch, about 0.35 us a
    tensor: the usual case takes one expression, the message is found after.)"""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and
                t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _check_device(t, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check_device(t, name, dev):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, expected {dev}")


def _rows(t, name, dtype, shape, dev):
    """(address, token stride) of rows of shape (tokens, heads, dim) whose heads lie side by
    side (columns of wider rows are accepted)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            n, heads, dim = shape
            st, sh, sd = t.stride()
            if sd == 1 and (sh == dim or heads == 1) or t.is_contiguous():
                return t.data_ptr(), (st if n > 1 else heads * dim)
            raise ValueError(f"{name}: the heads of a token must lie side by side "
                             f"(stride {t.stride()})")
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _check_device(t, name, dev)
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _device_of(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _stream(stream, dev):
    """cudaStream_t as an int: the device's current stream by default."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(dev)
        return torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != dev:
            raise ValueError(f"the stream is on device {stream.device_index}, the tensors on {dev}")
        return stream.cuda_stream
    return int(stream)


def _call(fn, dev, args):
    """fn(*args) with the tensors' device as the current one while it launches."""
    if torch.cuda.current_device() == dev:
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status != PA_OK:
        raise PAError(fn.__name__, status)


def _answer(fn, status):
    """Whether the extension made the call; raises for a status."""
    if status is None:
        return False
    if status != PA_OK:
        raise PAError(fn, status)
    return True


def _error_ptr(t, dev):
    """Address of a device error word: the first 4 bytes of `t` (None: not wanted)."""
    if t is None:
        return None
    _check_device(t, "device_error", dev)
    if t.numel() * t.element_size() < 4 or not t.is_contiguous():
        raise ValueError("device_error must hold 4 contiguous bytes")
    return t.data_ptr()


def pa_q4_page_bytes(head_dim: int) -> int:
    """Bytes of one (page, KV head) block; 0 for a head_dim that is not supported."""
    return _lib().pa_q4_page_bytes(int(head_dim))


def new_q4_cache(num_pages, num_kv_heads, head_dim, device=None) -> torch.Tensor:
    """Zero-filled 4-bit cache (every code then stands for 0)."""
    n = pa_q4_page_bytes(head_dim)
    if n == 0:
        raise ValueError(f"head_dim {head_dim} is not supported")
    return torch.zeros((num_pages, num_kv_heads, n), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def _cache_dims(cache, dev, head_dim):
    if not isinstance(cache, torch.Tensor):
        raise TypeError("cache must be a torch.Tensor")
    if cache.dtype != torch.uint8:
        raise TypeError(f"cache must be torch.uint8, got {cache.dtype}")
    if cache.dim() != 3 or cache.shape[2] != 20 * head_dim:
        raise ValueError(f"cache must have shape (num_pages, Hkv, {20 * head_dim}), "
                         f"got {tuple(cache.shape)}")
    _check_device(cache, "cache", dev)
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    return cache.shape[0], cache.shape[1]


def _cache_args(k, v, slots, cache):
    dev = _device_of(k, "k")
    if k.dim() != 3:
        raise ValueError(f"k must have shape (tokens, Hkv, D), got {tuple(k.shape)}")
    n, _, dim = k.shape
    et = k.dtype
    if et not in _DTYPE:
        raise TypeError(f"k must be fp16 or bf16, got {et}")
    pages, hkv = _cache_dims(cache, dev, dim)
    shape = (n, hkv, dim)
    return (dev, (n, hkv, dim, PAGE_SIZE, pages, _DTYPE[et]), _rows(k, "k", et, shape, dev),
            _rows(v, "v", et, shape, dev), _check(slots, "slots", torch.int64, (n,), dev),
            cache.data_ptr())


def pa_q4_write(k, v, slots, cache, device_error=None, stream=None) -> None:
    """Quantise rows k, v [tokens, Hkv, D] (fp16 or bf16, columns of wider rows allowed)
    into the cache at `slots` (int64 [tokens], distinct; -1: left out)."""
    if _fast is not None and device_error is None and stream is None and _answer(
            "pa_q4_write", _fast.q4_write(k, v, slots, cache)):
        return
    dev, sizes, kr, vr, sl, cp = _cache_args(k, v, slots, cache)
    _call(_lib().pa_q4_write, dev, (*sizes, *kr, *vr, sl, cp, _error_ptr(device_error, dev),
                                    _stream(stream, dev)))


def pa_q4_read(cache, slots, k_out, v_out, device_error=None, stream=None) -> None:
    """Rows the cache stands for at `slots`, into k_out, v_out [tokens, Hkv, D]
    (slot -1: zeros)."""
    if _fast is not None and device_error is None and stream is None and _answer(
            "pa_q4_read", _fast.q4_read(cache, slots, k_out, v_out)):
        return
    dev, sizes, kr, vr, sl, cp = _cache_args(k_out, v_out, slots, cache)
    _call(_lib().pa_q4_read, dev, (*sizes, cp, sl, *kr, *vr, _error_ptr(device_error, dev),
                                   _stream(stream, dev)))


def pa_q4_plan(batch, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
               max_pages_per_seq, max_context_len, window=0, num_sms=0,
               dtype=PA_DTYPE_F16) -> pa_q4_plan_t:
    """Plan decode calls over a 4-bit cache (num_sms 0: ask the current device)."""
    plan = pa_q4_plan_t()
    st = _lib().pa_q4_plan(
        int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size),
        int(num_pages), int(max_pages_per_seq), int(max_context_len), int(window), int(num_sms),
        int(dtype), ctypes.byref(plan))
    if st != PA_OK:
        raise PAError("pa_q4_plan", st)
    return plan


def _q4_decode_args(plan, q, cache, block_tables, context_lens, scale, window, out, lse,
                    workspace, stream):
    et = _TORCH.get(plan.dtype, torch.float16)
    dev = _device_of(q, "q")
    B, Hq, D = plan.batch, plan.num_q_heads, plan.head_dim
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    _check_device(workspace, "workspace", dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.numel() * workspace.element_size() < plan.workspace_bytes:
        raise PAError("pa_q4_decode", 4)
    return dev, (ctypes.byref(plan), _check(q, "q", et, (B, Hq, D), dev),
                 _check(cache, "cache", torch.uint8,
                        (plan.num_pages, plan.num_kv_heads, 20 * D), dev),
                 _check(block_tables, "block_tables", torch.int32,
                        (B, plan.max_pages_per_seq), dev),
                 _check(context_lens, "context_lens", torch.int32, (B,), dev),
                 float(scale), int(window), _check(out, "out", et, (B, Hq, D), dev),
                 _check(lse, "lse", torch.float32, (B, Hq), dev), workspace.data_ptr(),
                 _stream(stream, dev))


def pa_q4_decode(plan, q, cache, block_tables, context_lens, scale, window, out, lse, workspace,
                 stream=None) -> None:
    """One decode step over a 4-bit cache; arguments as pa_decode's."""
    if _fast is not None and stream is None and _answer(
            "pa_q4_decode", _fast.q4_decode(plan, q, cache, block_tables, context_lens, scale,
                                            window, out, lse, workspace)):
        return
    dev, args = _q4_decode_args(plan, q, cache, block_tables, context_lens, scale, window, out,
                                lse, workspace, stream)
    _call(_lib().pa_q4_decode, dev, args)


class PreparedQ4Decode:
    """pa_q4_decode with its arguments checked and converted once, for a loop that
    calls it with the same buffers every step (as PreparedDecode for pa_decode).
    The tensors must stay alive and in place while it is used.  Every call goes to
    the stream of the preparation: `stream`, or without one the stream that was
    current then (prepare inside torch.cuda.graph what a graph is to capture)."""

    def __init__(self, plan, q, cache, block_tables, context_lens, scale, window, out, lse,
                 workspace, stream=None):
        self.plan = pa_q4_plan_t.from_buffer_copy(plan)
        self._keep = (q, cache, block_tables, context_lens, out, lse, workspace)
        self._dev, self._args = _q4_decode_args(self.plan, q, cache, block_tables, context_lens,
                                                scale, window, out, lse, workspace, stream)
        self._fn = _lib().pa_q4_decode

    def __call__(self) -> None:
        _call(self._fn, self._dev, self._args)


def prepare_q4_decode(plan, q, cache, block_tables, context_lens, scale, window, out, lse,
                      workspace, stream=None) -> PreparedQ4Decode:
    """Check and convert pa_q4_decode's arguments once; calling the result launches."""
    return PreparedQ4Decode(plan, q, cache, block_tables, context_lens, scale, window, out, lse,
                            workspace, stream)


def q4_decode(q, cache, block_tables, context_lens, scale, window=0, max_context_len=None,
              stream=None):
    """Convenience call: plan, allocate out/lse/workspace with torch, decode.

    Returns (out, lse, plan, device_error); device_error is read back, so this
    call synchronises."""
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"q must be fp16 or bf16, got {q.dtype}")
    dev = _device_of(q, "q")
    B, Hq, D = q.shape
    pages, hkv = _cache_dims(cache, dev, D)
    maxp = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxp * PAGE_SIZE
    with torch.cuda.device(dev):
        plan = pa_q4_plan(B, Hq, hkv, D, PAGE_SIZE, pages, maxp, max_context_len, window, 0,
                          _DTYPE[q.dtype])
        st = _stream(stream, dev)
        out = torch.empty((B, Hq, D), dtype=q.dtype, device=q.device)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
        ws = new_workspace(plan, q.device)
        if stream is not None:  # the workspace is zeroed on the current stream
            torch.cuda.current_stream(dev).synchronize()
        pa_q4_decode(plan, q, cache, block_tables, context_lens, scale, window, out, lse, ws, st)
        err = pa_get_error(ws, st)
    return out, lse, plan, err


def pa_extend_tables(past_lens, new_lens, free_pages, num_pages, block_tables, context_lens,
                     starts, slots, positions, pages_taken, device_error=None,
                     stream=None) -> None:
    """Block tables, lengths, slots and positions of a step, from the requests' lengths
    (past_lens, new_lens int32 [B]) and a list of free pages (int32); see include/pa_q4.h."""
    if _fast is not None and device_error is None and stream is None and _answer(
            "pa_extend_tables", _fast.extend_tables(past_lens, new_lens, free_pages, num_pages,
                                                    block_tables, context_lens, starts, slots,
                                                    positions, pages_taken)):
        return
    dev = _device_of(past_lens, "past_lens")
    if block_tables.dim() != 2 or slots.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("block_tables must be 2-D, slots and free_pages 1-D")
    B, i32 = past_lens.shape[0], torch.int32
    maxp, cap, free = block_tables.shape[1], slots.shape[0], free_pages.shape[0]
    args = (B, maxp, PAGE_SIZE, int(num_pages), free, cap,
            _check(past_lens, "past_lens", i32, (B,), dev),
            _check(new_lens, "new_lens", i32, (B,), dev),
            _check(free_pages, "free_pages", i32, (free,), dev),
            _check(block_tables, "block_tables", i32, (B, maxp), dev),
            _check(context_lens, "context_lens", i32, (B,), dev),
            _check(starts, "starts", i32, (B + 1,), dev),
            _check(slots, "slots", torch.int64, (cap,), dev),
            _check(positions, "positions", i32, (cap,), dev),
            _check(pages_taken, "pages_taken", i32, (1,), dev),
            _error_ptr(device_error, dev), _stream(stream, dev))
    _call(_lib().pa_extend_tables, dev, args)


def pa_rope_axes(q, k, positions, sections, theta, q_out=None, k_out=None, rotary_dim=None,
                 interleaved=False, inverse=False, stream=None) -> None:
    """Rotary embedding of q [tokens, Hq, D] and k [tokens, Hkv, D] (fp16, bf16 or fp32,
    columns of wider rows allowed) with positions int32 [axes, tokens]; sections: pairs
    per axis.  q_out, k_out default to q and k (in place); q or k may be None.
    inverse=True turns back: applied to a gradient it is the rotation's backward pass."""
    if _fast is not None and stream is None and _answer(
            "pa_rope_axes", _fast.rope_axes(q, k, positions, sections, theta, q_out, k_out,
                                            rotary_dim, interleaved, inverse)):
        return
    some = q if q is not None else k
    if some is None:
        raise ValueError("q or k is needed")
    dev = _device_of(some, "q" if q is not None else "k")
    if some.dim() != 3:
        raise ValueError(f"q and k must have shape (tokens, heads, D), got {tuple(some.shape)}")
    n, _, D = some.shape
    et = some.dtype
    if et not in _DTYPE:
        raise TypeError(f"q and k must be fp16, bf16 or fp32, got {et}")
    axes = len(sections)
    hq = hk = 0
    qp = ks = qs = kp = qop = kop = qos = kos = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must have shape (tokens, heads, D), got {tuple(q.shape)}")
        hq = q.shape[1]
        qp, qs = _rows(q, "q", et, (n, hq, D), dev)
        qop, qos = (qp, qs) if q_out is None else _rows(q_out, "q_out", et, (n, hq, D), dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        if k.dim() != 3:
            raise ValueError(f"k must have shape (tokens, heads, D), got {tuple(k.shape)}")
        hk = k.shape[1]
        kp, ks = _rows(k, "k", et, (n, hk, D), dev)
        kop, kos = (kp, ks) if k_out is None else _rows(k_out, "k_out", et, (n, hk, D), dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    args = (n, hq, hk, D, D if rotary_dim is None else int(rotary_dim), axes,
            (ctypes.c_int * axes)(*sections), 1 if interleaved else 0, 1 if inverse else 0,
            float(theta), _DTYPE[et], qp or None, qs, kp or None, ks,
            _check(positions, "positions", torch.int32, (axes, n), dev), qop or None, qos,
            kop or None, kos, _stream(stream, dev))
    _call(_lib().pa_rope_axes, dev, args)
