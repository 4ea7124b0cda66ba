"""The operators of include/pa_q8.h over torch CUDA tensors.

Every function checks its tensors, converts them to pointers and calls the C
ABI of the same name on the tensors' device and a stream of it (the current
one by default); all computation runs in the library's CUDA kernels.  Outputs
are written into tensors the caller passes, nothing is allocated, and no call
synchronises (the convenience call ``q8_decode`` does both).

An 8-bit cache is a pair of torch.float8_e4m3fn tensors [num_pages, Hkv, 16, D]
for K and V and a pair of float32 tensors [num_pages, Hkv] of their scales
(``new_q8_cache``): a code stands for its value times the scale of its page and
KV head.
"""
from __future__ import annotations

import ctypes

import torch

from . import q4 as _q4
from .binding import PA_DTYPE_F16, PA_OK, PAError, new_workspace, pa_get_error
from .q4 import (_DTYPE, _TORCH, PAGE_SIZE, _answer, _call, _check, _check_device, _device_of,
                 _error_ptr, _rows, _stream)

PA_DEVERR_BAD_TOKEN = 32
PA_VERIFY_MAX_DRAFTS = 32
_F8 = torch.float8_e4m3fn


class pa_q8_plan_t(ctypes.Structure):
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
        ("max_query_len", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("num_sms", ctypes.c_int),
        ("heads_per_cta", ctypes.c_int),
        ("ctas_per_group", ctypes.c_int),
        ("ctas", ctypes.c_int),
        ("ctrl_bytes", ctypes.c_int),
        ("workspace_bytes", ctypes.c_size_t),
        ("test_stall_bytes", ctypes.c_int),
        ("cluster", ctypes.c_int),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


_bound = None


def _lib():
    """The library with this module's signatures set."""
    global _bound
    if _bound is not None:
        return _bound
    lib = _q4._lib()
    P, i, ll, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    plan = ctypes.POINTER(pa_q8_plan_t)
    rows = [i] * 8 + [f, f] + [P, ll] * 3 + [P] * 5 + [ll, P, P]
    lib.pa_append.argtypes = rows + [P, P]
    lib.pa_append.restype = i
    lib.pa_q8_append.argtypes = rows + [P] * 4
    lib.pa_q8_append.restype = i
    lib.pa_q8_read.argtypes = [i] * 6 + [P] * 5 + [P, ll, P, ll, P, P]
    lib.pa_q8_read.restype = i
    lib.pa_q8_plan.argtypes = [i] * 12 + [plan]
    lib.pa_q8_plan.restype = i
    lib.pa_q8_decode.argtypes = [plan, i] + [P] * 8 + [f, i] + [P] * 4
    lib.pa_q8_decode.restype = i
    lib.pa_verify_drafts.argtypes = [i] * 4 + [P] * 10
    lib.pa_verify_drafts.restype = i
    if _q4._fast is not None:
        names = ("pa_append", "pa_q8_append", "pa_q8_read", "pa_q8_decode", "pa_verify_drafts")
        _q4._fast.setup_q8(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                                 for n in names))
    _bound = lib
    return lib


def _fast():
    """The marshalling extension (as q4.py's), once the library is loaded."""
    return _q4._fast if _bound is not None else None


def new_q8_cache(num_pages, num_kv_heads, head_dim, device=None):
    """(k_cache, v_cache, k_scales, v_scales) of an empty 8-bit cache: codes of 0, scales 1."""
    if head_dim not in (64, 96, 128, 256):
        raise ValueError(f"head_dim {head_dim} is not supported")
    dev = "cuda" if device is None else device
    shape = (num_pages, num_kv_heads, PAGE_SIZE, head_dim)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device=dev).view(_F8) for _ in range(2))
    ks, vs = (torch.ones(shape[:2], dtype=torch.float32, device=dev) for _ in range(2))
    return k, v, ks, vs


def _cache_dims(t, name, dtype, dev, heads, dim):
    """Pages of a cache [pages, heads, 16, dim]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must have shape (num_pages, Hkv, {PAGE_SIZE}, D), "
                         f"got {tuple(t.shape)}")
    return t.shape[0], _check(t, name, dtype, (t.shape[0], heads, PAGE_SIZE, dim), dev)


def _three(t, name):
    dev = _device_of(t, name)
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape (tokens, heads, D), got {tuple(t.shape)}")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name} must be fp16, bf16 or fp32, got {t.dtype}")
    return dev


def _append_args(q, k, v, slots, positions, k_cache, v_cache, q_out, q_norm, k_norm, eps, theta,
                 rotary_dim, cache_dtype):
    dev = _three(k, "k")
    n, hkv, D = k.shape
    et = k.dtype
    kp, ks = _rows(k, "k", et, (n, hkv, D), dev)
    vp, vs = _rows(v, "v", et, (n, hkv, D), dev)
    hq = qs = qos = 0
    qp = qop = qn = None
    if q is not None:
        _three(q, "q")
        hq = q.shape[1]
        qp, qs = _rows(q, "q", et, (n, hq, D), dev)
        qop, qos = (qp, qs) if q_out is None else _rows(q_out, "q_out", et, (n, hq, D), dev)
        if q_norm is not None:
            qn = _check(q_norm, "q_norm", et, (D,), dev)
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out or q_norm without q")
    kn = None if k_norm is None else _check(k_norm, "k_norm", et, (D,), dev)
    theta = float(theta)
    pos = None
    if theta != 0.0:
        pos = _check(positions, "positions", torch.int32, (n,), dev)
    ct = et if cache_dtype is None else cache_dtype
    pages, kc = _cache_dims(k_cache, "k_cache", ct, dev, hkv, D)
    vc = _check(v_cache, "v_cache", ct, (pages, hkv, PAGE_SIZE, D), dev)
    sl = _check(slots, "slots", torch.int64, (n,), dev)
    return dev, (pages, hkv), (
        n, hq, hkv, D, D if rotary_dim is None else int(rotary_dim), PAGE_SIZE, pages,
        _DTYPE[et], theta, float(eps), qp, qs, kp, ks, vp, vs, qn, kn, pos, sl, qop, qos, kc, vc)


def pa_append(q, k, v, slots, positions, k_cache, v_cache, q_out=None, q_norm=None, k_norm=None,
              eps=1e-6, theta=0.0, rotary_dim=None, device_error=None, stream=None) -> None:
    """New rows q [tokens, Hq, D], k, v [tokens, Hkv, D] (fp16, bf16 or fp32, columns of wider
    rows allowed): heads of q and k normalised (with the weights q_norm, k_norm [D], where given)
    and rotated (theta > 0, positions int32 [tokens]), q written to q_out (default: in place),
    k and v into the paged cache [num_pages, Hkv, 16, D] of their type at `slots` (int64
    [tokens], distinct; -1: left out).  q may be None."""
    if device_error is None and stream is None and (fast := _fast()) is not None and _answer(
            "pa_append", fast.append(q, k, v, slots, positions, k_cache, v_cache, q_out, q_norm,
                                     k_norm, eps, theta, rotary_dim)):
        return
    dev, _, args = _append_args(q, k, v, slots, positions, k_cache, v_cache, q_out, q_norm,
                                k_norm, eps, theta, rotary_dim, None)
    _call(_lib().pa_append, dev, (*args, _error_ptr(device_error, dev), _stream(stream, dev)))


def pa_q8_append(q, k, v, slots, positions, k_cache, v_cache, k_scales, v_scales, q_out=None,
                 q_norm=None, k_norm=None, eps=1e-6, theta=0.0, rotary_dim=None,
                 device_error=None, stream=None) -> None:
    """pa_append into an 8-bit cache (``new_q8_cache``).  A page's rows lie next to one another
    among the tokens, at ascending slots; see include/pa_q8.h."""
    if device_error is None and stream is None and (fast := _fast()) is not None and _answer(
            "pa_q8_append", fast.q8_append(q, k, v, slots, positions, k_cache, v_cache, q_out,
                                           q_norm, k_norm, eps, theta, rotary_dim, k_scales,
                                           v_scales)):
        return
    dev, shape, args = _append_args(q, k, v, slots, positions, k_cache, v_cache, q_out, q_norm,
                                    k_norm, eps, theta, rotary_dim, _F8)
    _call(_lib().pa_q8_append, dev,
          (*args, _check(k_scales, "k_scales", torch.float32, shape, dev),
           _check(v_scales, "v_scales", torch.float32, shape, dev),
           _error_ptr(device_error, dev), _stream(stream, dev)))


def pa_q8_read(k_cache, v_cache, k_scales, v_scales, slots, k_out, v_out, device_error=None,
               stream=None) -> None:
    """Rows an 8-bit cache stands for at `slots`, into k_out, v_out [tokens, Hkv, D] (fp16, bf16
    or fp32; slot -1: zeros)."""
    if device_error is None and stream is None and (fast := _fast()) is not None and _answer(
            "pa_q8_read", fast.q8_read(k_cache, v_cache, k_scales, v_scales, slots, k_out, v_out)):
        return
    dev = _three(k_out, "k_out")
    n, hkv, D = k_out.shape
    et = k_out.dtype
    pages, kc = _cache_dims(k_cache, "k_cache", _F8, dev, hkv, D)
    args = (n, hkv, D, PAGE_SIZE, pages, _DTYPE[et], kc,
            _check(v_cache, "v_cache", _F8, (pages, hkv, PAGE_SIZE, D), dev),
            _check(k_scales, "k_scales", torch.float32, (pages, hkv), dev),
            _check(v_scales, "v_scales", torch.float32, (pages, hkv), dev),
            _check(slots, "slots", torch.int64, (n,), dev),
            *_rows(k_out, "k_out", et, (n, hkv, D), dev),
            *_rows(v_out, "v_out", et, (n, hkv, D), dev), _error_ptr(device_error, dev),
            _stream(stream, dev))
    _call(_lib().pa_q8_read, dev, args)


def pa_q8_plan(batch, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
               max_pages_per_seq, max_context_len, window=0, max_query_len=1, num_sms=0,
               dtype=PA_DTYPE_F16) -> pa_q8_plan_t:
    """Plan decode calls over an 8-bit cache (num_sms 0: ask the current device)."""
    plan = pa_q8_plan_t()
    st = _lib().pa_q8_plan(
        int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size),
        int(num_pages), int(max_pages_per_seq), int(max_context_len), int(window),
        int(max_query_len), int(num_sms), int(dtype), ctypes.byref(plan))
    if st != PA_OK:
        raise PAError("pa_q8_plan", st)
    return plan


def _q8_decode_args(plan, q, starts, k_cache, v_cache, k_scales, v_scales, block_tables,
                    context_lens, scale, window, out, lse, workspace, stream):
    et = _TORCH.get(plan.dtype, torch.float16)
    dev = _device_of(q, "q")
    B, Hq, D = plan.batch, plan.num_q_heads, plan.head_dim
    if q.dim() != 3:
        raise ValueError(f"q must have shape (rows, Hq, D), got {tuple(q.shape)}")
    n = q.shape[0]
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    _check_device(workspace, "workspace", dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.numel() * workspace.element_size() < plan.workspace_bytes:
        raise PAError("pa_q8_decode", 4)
    if starts is None and n < B:
        raise ValueError(f"q must have a row for each of {B} sequences, got {n}")
    cache = (plan.num_pages, plan.num_kv_heads, PAGE_SIZE, D)
    return dev, (ctypes.byref(plan), n, _check(q, "q", et, (n, Hq, D), dev),
                 None if starts is None else _check(starts, "starts", torch.int32, (B + 1,), dev),
                 _check(k_cache, "k_cache", _F8, cache, dev),
                 _check(v_cache, "v_cache", _F8, cache, dev),
                 _check(k_scales, "k_scales", torch.float32, cache[:2], dev),
                 _check(v_scales, "v_scales", torch.float32, cache[:2], dev),
                 _check(block_tables, "block_tables", torch.int32,
                        (B, plan.max_pages_per_seq), dev),
                 _check(context_lens, "context_lens", torch.int32, (B,), dev),
                 float(scale), int(window), _check(out, "out", et, (n, Hq, D), dev),
                 _check(lse, "lse", torch.float32, (n, Hq), dev), workspace.data_ptr(),
                 _stream(stream, dev))


def pa_q8_decode(plan, q, starts, k_cache, v_cache, k_scales, v_scales, block_tables,
                 context_lens, scale, window, out, lse, workspace, stream=None) -> None:
    """Attention of rows starts[b] .. starts[b + 1] - 1 of q [rows, Hq, D], sequence b's last
    tokens, over an 8-bit cache (starts int32 [B + 1], as pa_extend_tables makes them; None: one
    row per sequence); the other arguments as pa_decode's."""
    if stream is None and (fast := _fast()) is not None and _answer(
            "pa_q8_decode", fast.q8_decode(plan, q, starts, k_cache, v_cache, k_scales, v_scales,
                                           block_tables, context_lens, scale, window, out, lse,
                                           workspace)):
        return
    dev, args = _q8_decode_args(plan, q, starts, k_cache, v_cache, k_scales, v_scales,
                                block_tables, context_lens, scale, window, out, lse, workspace,
                                stream)
    _call(_lib().pa_q8_decode, dev, args)


class PreparedQ8Decode:
    """pa_q8_decode with its arguments checked and converted once, for a loop that
    calls it with the same buffers every step (as PreparedDecode for pa_decode).
    The tensors must stay alive and in place while it is used.  Every call goes to
    the stream of the preparation: `stream`, or without one the stream that was
    current then (prepare inside torch.cuda.graph what a graph is to capture)."""

    def __init__(self, plan, q, starts, k_cache, v_cache, k_scales, v_scales, block_tables,
                 context_lens, scale, window, out, lse, workspace, stream=None):
        self.plan = pa_q8_plan_t.from_buffer_copy(plan)
        self._keep = (q, starts, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                      out, lse, workspace)
        self._dev, self._args = _q8_decode_args(self.plan, q, starts, k_cache, v_cache, k_scales,
                                                v_scales, block_tables, context_lens, scale,
                                                window, out, lse, workspace, stream)
        self._fn = _lib().pa_q8_decode

    def __call__(self) -> None:
        _call(self._fn, self._dev, self._args)


def prepare_q8_decode(plan, q, starts, k_cache, v_cache, k_scales, v_scales, block_tables,
                      context_lens, scale, window, out, lse, workspace,
                      stream=None) -> PreparedQ8Decode:
    """Check and convert pa_q8_decode's arguments once; calling the result launches."""
    return PreparedQ8Decode(plan, q, starts, k_cache, v_cache, k_scales, v_scales, block_tables,
                            context_lens, scale, window, out, lse, workspace, stream)


def q8_decode(q, starts, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale,
              window=0, max_query_len=None, max_context_len=None, stream=None):
    """Convenience call: plan, allocate out/lse/workspace with torch, decode (rows that no
    sequence has: zeros).  max_query_len defaults to the longest of `starts`, which is read back.

    Returns (out, lse, plan, device_error); device_error is read back, so this
    call synchronises."""
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"q must be fp16 or bf16, got {q.dtype}")
    dev = _device_of(q, "q")
    n, Hq, D = q.shape
    B, maxp = block_tables.shape
    pages, hkv = k_cache.shape[:2]
    if max_context_len is None:
        max_context_len = maxp * PAGE_SIZE
    with torch.cuda.device(dev):
        st = _stream(stream, dev)
        if stream is not None:  # what is allocated here is filled on the current stream
            torch.cuda.ExternalStream(st, device=dev).synchronize()
        if max_query_len is None:
            max_query_len = 1
            if starts is not None and B > 0:
                max_query_len = max(1, int((starts[1:] - starts[:-1]).max()))
        plan = pa_q8_plan(B, Hq, hkv, D, PAGE_SIZE, pages, maxp, max_context_len, window,
                          max_query_len, 0, _DTYPE[q.dtype])
        out = torch.zeros((n, Hq, D), dtype=q.dtype, device=q.device)
        lse = torch.zeros((n, Hq), dtype=torch.float32, device=q.device)
        ws = new_workspace(plan, q.device)
        if stream is not None:
            torch.cuda.current_stream(dev).synchronize()
        pa_q8_decode(plan, q, starts, k_cache, v_cache, k_scales, v_scales, block_tables,
                     context_lens, scale, window, out, lse, ws, st)
        err = pa_get_error(ws, st)
    return out, lse, plan, err


def pa_verify_drafts(target_probs, draft_probs, draft_tokens, num_drafts, accept_u, sample_u,
                     accepted, tokens, device_error=None, stream=None) -> None:
    """Verification of drafted tokens (int32 [B, T]): accepted (int32 [B]) of them stand against
    target_probs [B, T + 1, V] and draft_probs [B, T, V] (None: certain drafts), and `tokens`
    (int32 [B, T + 1]) gets them, one drawn token and -1.  num_drafts int32 [B] (None: T each),
    random numbers accept_u [B, T] and sample_u [B] float32 of [0, 1); see include/pa_q8.h."""
    if device_error is None and stream is None and (fast := _fast()) is not None and _answer(
            "pa_verify_drafts", fast.verify(target_probs, draft_probs, draft_tokens, num_drafts,
                                            accept_u, sample_u, accepted, tokens)):
        return
    dev = _three(target_probs, "target_probs")
    B, T1, V = target_probs.shape
    T, et, i32, f32 = T1 - 1, target_probs.dtype, torch.int32, torch.float32
    args = (B, T, V, _DTYPE[et], _check(target_probs, "target_probs", et, (B, T1, V), dev),
            None if draft_probs is None else _check(draft_probs, "draft_probs", et, (B, T, V), dev),
            _check(draft_tokens, "draft_tokens", i32, (B, T), dev),
            None if num_drafts is None else _check(num_drafts, "num_drafts", i32, (B,), dev),
            _check(accept_u, "accept_u", f32, (B, T), dev),
            _check(sample_u, "sample_u", f32, (B,), dev),
            _check(accepted, "accepted", i32, (B,), dev),
            _check(tokens, "tokens", i32, (B, T1), dev), _error_ptr(device_error, dev),
            _stream(stream, dev))
    _call(_lib().pa_verify_drafts, dev, args)
