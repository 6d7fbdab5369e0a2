"""Causal kernelized linear attention for B200 (sm_100a).

Thin Python binding over the C ABI in ``include/la.h`` (``libla.so``, built
in-tree by ``causal_kernelized_linear_la_b200.build``).  This module only
marshals arguments: it checks devices, dtypes and shapes of torch tensors,
allocates outputs with torch, and passes raw device pointers and the current
CUDA stream to the library.  Every step of the computation runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback.  If libla.so is
missing or no GPU is present, calls raise.

Entry points (same names as the C ABI):

* ``la_prefill(q, k, v, mode=..., gamma=..., alpha=..., g=..., S0=..., z0=..., eps=...)``
  -> ``(o, S, z)`` (``z`` is None in gated-delta mode)
* ``la_prefill_varlen(q, k, v, seq_lens, mode=..., ...)`` -> ``(o, S, z)`` for a
  right-padded batch of sequences of different lengths
* ``la_decode_step(q, k, v, S, z, eps=...)`` -> ``o``; S and z updated in place
* ``la_gated_delta_decode_step(q, k, v, alpha, g, S)`` -> ``o``; S updated in place
* ``la_causal_conv(x, weight, cache)`` -> ``(out, cache_out)``
* ``la_ssm_conv(x, weight, bias=..., cache=..., silu=...)`` -> ``(out, cache_out)``,
  ``la_ssm_scan(x, delta, A, B, C, ...)`` -> ``(y, h)`` and
  ``la_ssm_step(x, delta, A, B, C, h, ...)`` -> ``y``: the convolution, prompt
  recurrence and token step of a selective state-space layer
* ``la_window_prefill(q, k, v, window, sinks=..., k_cache=..., v_cache=..., pos=...)``
  -> ``o`` and ``la_window_decode_step(q, k, v, k_cache, v_cache, pos, window, ...)``
  -> ``o``: sliding-window attention with sinks; the rolling caches are updated in place
* ``la_prefill_workspace_bytes(...)``, ``la_prefill_kernel_count(...)``,
  ``la_prefill_varlen_workspace_bytes(...)``,
  ``la_status_string(code)``, ``lib()``
"""
from __future__ import annotations

import contextlib
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libla.so")

LA_OK, LA_ERR_INVALID, LA_ERR_UNSUPPORTED, LA_ERR_ALIGN, LA_ERR_CUDA, LA_ERR_TIMEOUT, LA_ERR_WORKSPACE = range(7)
LA_F32, LA_BF16 = 0, 1
MODES = {"plain": 0, "decay": 1, "gated_delta": 2, "gla": 3}

# Symbols the library exports; the header include/la.h declares exactly these.
EXPORTS = ("la_prefill", "la_prefill_noalloc", "la_prefill_workspace_bytes", "la_prefill_kernel_count",
           "la_prefill_varlen",
           "la_prefill_varlen_workspace_bytes", "la_decode_step", "la_gated_delta_decode_step",
           "la_set_stage_events", "la_causal_conv", "la_selftest_wait_timeout",
           "la_ssm_conv", "la_ssm_scan", "la_ssm_scan_workspace_bytes", "la_ssm_step",
           "la_window_prefill", "la_window_decode_step",
           "la_prefill_check", "la_status_string", "la_version")


class LaConfig(ctypes.Structure):
    """Mirror of ``la_config`` in include/la.h."""
    _fields_ = [("dtype", ctypes.c_int), ("mode", ctypes.c_int), ("eps", ctypes.c_float),
                ("stream", ctypes.c_void_p), ("S0", ctypes.c_void_p), ("z0", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class LaSsmStrides(ctypes.Structure):
    """Mirror of ``la_ssm_strides`` in include/la.h."""
    _fields_ = [(f"{t}_{a}", ctypes.c_longlong) for t in ("x", "delta", "z", "B", "C") for a in ("batch", "row")]


class LaWindowStrides(ctypes.Structure):
    """Mirror of ``la_window_strides`` in include/la.h."""
    _fields_ = [(f"{t}_{a}", ctypes.c_longlong) for t in ("q", "k", "v", "out") for a in ("batch", "head", "row")]


class LaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {la_status_string(code)}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with causal_kernelized_linear_la_b200.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, cfgp = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(LaConfig)
        L.la_prefill.argtypes = [vp] * 8 + [i] * 5 + [cfgp]
        L.la_prefill.restype = i
        L.la_prefill_noalloc.argtypes = [vp] * 8 + [i] * 5 + [cfgp]
        L.la_prefill_noalloc.restype = i
        L.la_prefill_workspace_bytes.argtypes = [i] * 5 + [cfgp]
        L.la_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.la_prefill_kernel_count.argtypes = [i] * 5 + [cfgp]
        L.la_prefill_kernel_count.restype = i
        ip = ctypes.POINTER(ctypes.c_int)
        L.la_prefill_varlen.argtypes = [vp] * 8 + [ip] + [i] * 5 + [cfgp]
        L.la_prefill_varlen.restype = i
        L.la_prefill_varlen_workspace_bytes.argtypes = [ip] + [i] * 4 + [cfgp]
        L.la_prefill_varlen_workspace_bytes.restype = ctypes.c_size_t
        L.la_decode_step.argtypes = [vp] * 6 + [i] * 4 + [cfgp]
        L.la_decode_step.restype = i
        L.la_gated_delta_decode_step.argtypes = [vp] * 7 + [i] * 4 + [cfgp]
        L.la_gated_delta_decode_step.restype = i
        L.la_prefill_check.argtypes = [vp, vp]
        L.la_prefill_check.restype = i
        L.la_selftest_wait_timeout.argtypes = [vp]
        L.la_selftest_wait_timeout.restype = i
        L.la_causal_conv.argtypes = [vp] * 5 + [i] * 5 + [cfgp]
        L.la_causal_conv.restype = i
        ll, stp = ctypes.c_longlong, ctypes.POINTER(LaSsmStrides)
        L.la_ssm_conv.argtypes = [vp] * 6 + [ip] + [i] * 5 + [ll] * 2 + [cfgp]
        L.la_ssm_conv.restype = i
        L.la_ssm_scan.argtypes = [vp] * 10 + [ip] + [i] * 6 + [stp, cfgp]
        L.la_ssm_scan.restype = i
        L.la_ssm_scan_workspace_bytes.argtypes = [i] * 5
        L.la_ssm_scan_workspace_bytes.restype = ctypes.c_size_t
        L.la_ssm_step.argtypes = [vp] * 10 + [i] * 5 + [stp, cfgp]
        L.la_ssm_step.restype = i
        wsp, fl = ctypes.POINTER(LaWindowStrides), ctypes.c_float
        L.la_window_prefill.argtypes = [vp] * 7 + [ip] + [i] * 8 + [fl, wsp, cfgp]
        L.la_window_prefill.restype = i
        L.la_window_decode_step.argtypes = [vp] * 7 + [i] * 7 + [fl, wsp, cfgp]
        L.la_window_decode_step.restype = i
        L.la_set_stage_events.argtypes = [ctypes.POINTER(vp), i]
        L.la_set_stage_events.restype = i
        L.la_status_string.argtypes = [i]
        L.la_status_string.restype = ctypes.c_char_p
        L.la_version.argtypes = []
        L.la_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def la_status_string(code: int) -> str:
    return lib().la_status_string(int(code)).decode()


def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _check_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (the library has no CPU path)")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def _stream_handle(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def la_prefill_workspace_bytes(B, H, N, d, dv, dtype="bf16", mode="plain") -> int:
    cfg = LaConfig(LA_BF16 if dtype == "bf16" else LA_F32, MODES[mode], 0.0, None, None, None, None, 0)
    return int(lib().la_prefill_workspace_bytes(B, H, N, d, dv, ctypes.byref(cfg)))


def la_prefill_kernel_count(B, H, N, d, dv, dtype="bf16", mode="plain") -> int:
    """Kernels one la_prefill call with these sizes launches (host-only)."""
    cfg = LaConfig(LA_BF16 if dtype == "bf16" else LA_F32, MODES[mode], 0.0, None, None, None, None, 0)
    return int(lib().la_prefill_kernel_count(B, H, N, d, dv, ctypes.byref(cfg)))


def la_prefill(q, k, v, mode="plain", gamma=None, alpha=None, g=None, S0=None, z0=None, eps=1e-6,
               out=None, S_out=None, z_out=None, workspace=None, stream=None):
    """Causal prefill over [B,H,N,*] tensors; returns ``(o, S_N, z_N)``.

    mode "plain" (gamma = 1), "decay" (gamma [H] fp32), "gated_delta"
    (alpha, g [B,H,N] fp32; k L2-normalised; returns z_N = None), or "gla"
    (alpha [B,H,N,d] fp32, the per-key-channel gate; returns z_N = None)."""
    torch = _torch()
    if mode not in MODES:
        raise ValueError(f"mode must be one of {list(MODES)}")
    B, H, N, d = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, N) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k must be [B,H,N,d] and v [B,H,N,dv], all of one dtype")
    delta = mode in ("gated_delta", "gla")   # the modes without a normaliser
    dev = q.device
    if out is None:
        out = torch.empty((B, H, N, dv), device=dev, dtype=q.dtype)
    if S_out is None:
        S_out = torch.empty((B, H, d, dv), device=dev, dtype=torch.float32)
    if not delta and z_out is None:
        z_out = torch.empty((B, H, d), device=dev, dtype=torch.float32)
    if delta:
        z_out = None
    first = alpha if delta else gamma
    for t in (first, g, S0, z0, S_out, z_out):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("gamma/alpha/g/S0/z0/S_out/z_out must be float32")
    _check_cuda(q, k, v, first, g, S0, z0, out, S_out, z_out, workspace)
    need = la_prefill_workspace_bytes(B, H, N, d, dv, "bf16" if q.dtype == torch.bfloat16 else "f32", mode)
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    cfg = LaConfig(_dtype_code(q), MODES[mode], float(eps), _stream_handle(stream), _ptr(S0), _ptr(z0),
                   _ptr(workspace), ws_bytes)
    rc = lib().la_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(first), _ptr(g), _ptr(out), _ptr(S_out), _ptr(z_out),
                          B, H, N, d, dv, ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_prefill")
    return out, S_out, z_out


def _host_lens(seq_lens):
    """The sequence lengths as a C int array (host memory)."""
    lens = [int(n) for n in (seq_lens.tolist() if hasattr(seq_lens, "tolist") else seq_lens)]
    return (ctypes.c_int * max(len(lens), 1))(*lens), len(lens)


def la_prefill_varlen_workspace_bytes(seq_lens, H, d, dv, dtype="bf16", mode="plain") -> int:
    arr, B = _host_lens(seq_lens)
    cfg = LaConfig(LA_BF16 if dtype == "bf16" else LA_F32, MODES[mode], 0.0, None, None, None, None, 0)
    return int(lib().la_prefill_varlen_workspace_bytes(arr, B, H, d, dv, ctypes.byref(cfg)))


def la_prefill_varlen(q, k, v, seq_lens, mode="plain", gamma=None, alpha=None, g=None, S0=None, z0=None,
                      eps=1e-6, out=None, S_out=None, z_out=None, workspace=None, stream=None):
    """Prefill of a right-padded batch: q, k [B,H,N,d], v [B,H,N,dv] with
    sequence b in rows 0..seq_lens[b]-1 (seq_lens: host ints).  Returns
    ``(o, S, z)`` with each sequence's final state; rows of o past a
    sequence's length are not written (uninitialised when o is allocated
    here).  Other arguments as in ``la_prefill``."""
    torch = _torch()
    if mode not in MODES:
        raise ValueError(f"mode must be one of {list(MODES)}")
    B, H, N, d = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, N) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k must be [B,H,N,d] and v [B,H,N,dv], all of one dtype")
    arr, nl = _host_lens(seq_lens)
    if nl != B:
        raise ValueError(f"seq_lens has {nl} entries for a batch of {B}")
    delta = mode in ("gated_delta", "gla")   # the modes without a normaliser
    dev = q.device
    if out is None:
        out = torch.empty((B, H, N, dv), device=dev, dtype=q.dtype)
    if S_out is None:
        S_out = torch.empty((B, H, d, dv), device=dev, dtype=torch.float32)
    if not delta and z_out is None:
        z_out = torch.empty((B, H, d), device=dev, dtype=torch.float32)
    if delta:
        z_out = None
    first = alpha if delta else gamma
    for t in (first, g, S0, z0, S_out, z_out):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("gamma/alpha/g/S0/z0/S_out/z_out must be float32")
    _check_cuda(q, k, v, first, g, S0, z0, out, S_out, z_out, workspace)
    cfg = LaConfig(_dtype_code(q), MODES[mode], float(eps), _stream_handle(stream), _ptr(S0), _ptr(z0), None, 0)
    need = int(lib().la_prefill_varlen_workspace_bytes(arr, B, H, d, dv, ctypes.byref(cfg)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    cfg.workspace = _ptr(workspace)
    cfg.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().la_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(first), _ptr(g), _ptr(out), _ptr(S_out),
                                 _ptr(z_out), arr, B, H, N, d, dv, ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_prefill_varlen")
    return out, S_out, z_out


def la_decode_step(q, k, v, S, z, eps=1e-6, out=None, stream=None):
    """One decode step; q,k [B,H,d], v [B,H,dv]; S [B,H,d,dv], z [B,H,d]
    (fp32, updated in place).  Returns o [B,H,dv]."""
    torch = _torch()
    B, H, d = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, dv), device=q.device, dtype=q.dtype)
    _check_cuda(q, k, v, S, z, out)
    cfg = LaConfig(_dtype_code(q), MODES["plain"], float(eps), _stream_handle(stream), None, None, None, 0)
    rc = lib().la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(S), _ptr(z), _ptr(out), B, H, d, dv,
                              ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_decode_step")
    return out


def la_gated_delta_decode_step(q, k, v, alpha, g, S, out=None, stream=None):
    """One gated-delta decode step; alpha, g [B,H] fp32; S updated in place."""
    torch = _torch()
    B, H, d = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, dv), device=q.device, dtype=q.dtype)
    _check_cuda(q, k, v, alpha, g, S, out)
    cfg = LaConfig(_dtype_code(q), MODES["gated_delta"], 0.0, _stream_handle(stream), None, None, None, 0)
    rc = lib().la_gated_delta_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(g), _ptr(S), _ptr(out),
                                          B, H, d, dv, ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_gated_delta_decode_step")
    return out


def la_causal_conv(x, weight, cache=None, out=None, cache_out=None, stream=None):
    """Short causal convolution with conv cache on device tensors.
    x [B,H,N,d] bf16/fp32, weight [H,d,w] fp32, cache [B,H,w-1,d] or None.
    Returns (out, cache_out); cache_out is allocated when not given."""
    if x.dim() != 4 or weight.dim() != 3:
        raise ValueError("x must be [B,H,N,d] and weight [H,d,w]")
    torch = _torch()
    B, H, N, d = x.shape
    w = weight.shape[-1]
    if weight.shape != (H, d, w) or weight.dtype != torch.float32:
        raise ValueError("weight must be fp32 [H,d,w]")
    dev = x.device
    if out is None:
        out = torch.empty_like(x)
    if cache_out is None and w > 1:
        cache_out = torch.empty((B, H, w - 1, d), device=dev, dtype=x.dtype)
    _check_cuda(x, weight, cache, out, cache_out)
    cfg = LaConfig(_dtype_code(x), 0, 0.0, _stream_handle(stream), None, None, None, 0)
    rc = lib().la_causal_conv(_ptr(x), _ptr(weight), _ptr(cache), _ptr(out), _ptr(cache_out),
                              B, H, N, d, w, ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_causal_conv")
    return out, cache_out


def _on_device(first, others, stream):
    """Checks that every tensor is on the first one's CUDA device; returns that
    device's (given or current) stream handle and the device guard of the call."""
    cuda = _torch().cuda
    dev = first.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors (the library has no CPU path)")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"all tensors must be on one CUDA device, got {first.device} and {t.device}")
    if stream is None:
        # the handle alone where torch offers it: half the cost of a Stream object
        raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
        handle = raw(dev) if raw is not None else cuda.current_stream(dev).cuda_stream
    elif stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {first.device}")
    else:
        handle = stream.cuda_stream
    return handle, _NO_GUARD if dev == cuda.current_device() else cuda.device(dev)


_NO_GUARD = contextlib.nullcontext()


def _new(shape, dtype, dev, stream):
    """An output or workspace of a call on ``stream``: it comes from that
    stream's pool, so that memory still in use elsewhere is not handed out."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, device=dev, dtype=dtype)
    with torch.cuda.stream(stream):
        return torch.empty(shape, device=dev, dtype=dtype)


def _dense(t, shape, dtype, name):
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _addr(t):
    return None if t is None else t.data_ptr()


def _group_of(t, lead, D, name):
    """(G, n, batch stride, row stride) of B or C given as [*lead, n] or [*lead, G, n]."""
    shape, stride, k = t.shape, t.stride(), len(lead)
    if len(shape) == k + 1:
        G, n = 1, shape[k]
    elif len(shape) == k + 2:
        G, n = shape[k], shape[k + 1]
        if G > 1 and stride[k] != n:
            raise ValueError(f"the G * n values of a row of {name} must be contiguous")
    else:
        G = n = 0
    if n == 0 or shape[:k] != lead:
        raise ValueError(f"{name} must be [{', '.join(map(str, lead))}, G, n] (or without G), got {list(shape)}")
    if n > 1 and stride[-1] != 1:
        raise ValueError(f"the G * n values of a row of {name} must be contiguous")
    if G == 0 or D % G:
        raise ValueError(f"{name} has {G} groups for {D} channels")
    # an axis of one entry has no stride that matters
    return G, n, stride[0] if shape[0] > 1 else 0, stride[1] if k > 1 and shape[1] > 1 else 0


def _row_stride(t, name):
    """(batch stride, row stride) of [B, D] or [B, N, D]."""
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return stride[0] if shape[0] > 1 else 0, stride[1] if len(shape) > 2 and shape[1] > 1 else 0


def _lens_of(seq_lens, B):
    if seq_lens is None:
        return None
    arr, nl = _host_lens(seq_lens)
    if nl != B:
        raise ValueError(f"seq_lens has {nl} entries for a batch of {B}")
    return arr


def la_ssm_conv(x, weight, bias=None, cache=None, silu=True, seq_lens=None, out=None, cache_out=None, stream=None):
    """Short causal convolution of a state-space layer: x [B,N,D] bf16/fp32
    (batches and rows may be strided), weight [D,w] fp32, bias [D] fp32, cache
    [B,w-1,D] (the previous inputs; None: zero), seq_lens host ints of a
    right-padded batch.  Returns ``(out, cache_out)``; cache_out is allocated
    when not given and may be the cache itself.  One new token is N = 1."""
    torch = _torch()
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B,N,D] and weight [D,w]")
    B, N, D = x.shape
    w = weight.shape[1]
    xb, xt = _row_stride(x, "x")
    _dense(weight, (D, w), torch.float32, "weight")
    if bias is not None:
        _dense(bias, (D,), torch.float32, "bias")
    if out is None:
        out = _new((B, N, D), x.dtype, x.device, stream)
    if cache_out is None:
        cache_out = _new((B, w - 1, D), x.dtype, x.device, stream)
    _dense(out, (B, N, D), x.dtype, "out")
    _dense(cache_out, (B, w - 1, D), x.dtype, "cache_out")
    if cache is not None:
        _dense(cache, (B, w - 1, D), x.dtype, "cache")
    cfg = LaConfig(_dtype_code(x), 0, 0.0, None, None, None, None, 0)
    cfg.stream, guard = _on_device(x, (weight, bias, cache, out, cache_out), stream)
    with guard:
        rc = lib().la_ssm_conv(_addr(x), _addr(weight), _addr(bias), _addr(cache), _addr(out), _addr(cache_out),
                               _lens_of(seq_lens, B), B, N, D, w, int(silu), xb, xt, ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_ssm_conv")
    return out, cache_out


def la_ssm_scan_workspace_bytes(B, N, D, G, n) -> int:
    return int(lib().la_ssm_scan_workspace_bytes(B, N, D, G, n))


def _ssm_checks(x, delta, A, B, C, D, z, delta_bias):
    """Shapes and strides shared by the prompt scan and the token step."""
    torch = _torch()
    shape, dtype = x.shape, x.dtype
    ch = shape[-1]
    if delta.shape != shape or (z is not None and z.shape != shape):
        raise ValueError(f"delta and z must have the shape of x, {list(shape)}")
    G, n, Bb, Br = _group_of(B, shape[:-1], ch, "B")
    G2, n2, Cb, Cr = _group_of(C, shape[:-1], ch, "C")
    if G != G2 or n != n2:
        raise ValueError(f"B and C differ: {G} x {n} and {G2} x {n2}")
    if not (delta.dtype == dtype and B.dtype == dtype and C.dtype == dtype and (z is None or z.dtype == dtype)):
        raise ValueError("x, delta, B, C and z must have one dtype")
    _dense(A, (ch, n), torch.float32, "A")
    if D is not None:
        _dense(D, (ch,), torch.float32, "D")
    if delta_bias is not None:
        _dense(delta_bias, (ch,), torch.float32, "delta_bias")
    xb, xr = _row_stride(x, "x")
    db, dr = _row_stride(delta, "delta")
    zb, zr = _row_stride(z, "z") if z is not None else (0, 0)
    return G, n, LaSsmStrides(xb, xr, db, dr, zb, zr, Bb, Br, Cb, Cr)


def la_ssm_scan(x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False, h0=None, seq_lens=None,
                out=None, h_out=None, workspace=None, stream=None):
    """Selective state-space recurrence over prompts: x, delta, z [b,N,ch],
    B, C [b,N,G,n] or [b,N,n] (bf16/fp32, one dtype, rows may be strided), A
    [ch,n], D, delta_bias [ch] fp32, h0 [b,ch,n] fp32 start states, seq_lens host
    ints of a right-padded batch.  Returns ``(y, h)`` with the final states."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [B,N,D]")
    b, N, ch = x.shape
    G, n, st = _ssm_checks(x, delta, A, B, C, D, z, delta_bias)
    if out is None:
        out = _new((b, N, ch), x.dtype, x.device, stream)
    if h_out is None:
        h_out = _new((b, ch, n), torch.float32, x.device, stream)
    _dense(out, (b, N, ch), x.dtype, "out")
    _dense(h_out, (b, ch, n), torch.float32, "h_out")
    if h0 is not None:
        _dense(h0, (b, ch, n), torch.float32, "h0")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    cfg = LaConfig(_dtype_code(x), 0, 0.0, None, _addr(h0), None, None, 0)
    cfg.stream, guard = _on_device(x, (delta, A, B, C, D, z, delta_bias, h0, out, h_out, workspace), stream)
    need = la_ssm_scan_workspace_bytes(b, N, ch, G, n)
    if workspace is None and need > 0:
        workspace = _new(need, torch.uint8, x.device, stream)
    if workspace is not None:
        cfg.workspace = workspace.data_ptr()
        cfg.workspace_bytes = workspace.numel() * workspace.element_size()
    with guard:
        rc = lib().la_ssm_scan(_addr(x), _addr(delta), _addr(A), _addr(B), _addr(C), _addr(D), _addr(z),
                               _addr(delta_bias), _addr(out), _addr(h_out), _lens_of(seq_lens, b), b, N, ch, G, n,
                               int(delta_softplus), ctypes.byref(st), ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_ssm_scan")
    return out, h_out


def la_ssm_step(x, delta, A, B, C, h, D=None, z=None, delta_bias=None, delta_softplus=False, out=None, stream=None):
    """One token of each sequence: x, delta, z [b,ch]; B, C [b,G,n] or [b,n];
    h [b,ch,n] fp32 is updated in place.  Other arguments as in
    ``la_ssm_scan``.  Returns y [b,ch]."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [B,D]")
    b, ch = x.shape
    G, n, st = _ssm_checks(x, delta, A, B, C, D, z, delta_bias)
    if out is None:
        out = _new((b, ch), x.dtype, x.device, stream)
    _dense(out, (b, ch), x.dtype, "out")
    _dense(h, (b, ch, n), torch.float32, "h")
    cfg = LaConfig(_dtype_code(x), 0, 0.0, None, None, None, None, 0)
    cfg.stream, guard = _on_device(x, (delta, A, B, C, D, z, delta_bias, h, out), stream)
    with guard:
        rc = lib().la_ssm_step(_addr(x), _addr(delta), _addr(A), _addr(B), _addr(C), _addr(D), _addr(z),
                               _addr(delta_bias), _addr(h), _addr(out), b, ch, G, n, int(delta_softplus),
                               ctypes.byref(st), ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_ssm_step")
    return out


_INT = 1 << 31


def _head_strides(t, rows, name):
    """(batch, head, row) strides of [B, H, N, .] (rows) or [B, H, .]; an axis of one entry has none that matters."""
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return (stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0,
            stride[2] if rows and shape[2] > 1 else 0)


def _window_checks(q, k, v, out, k_cache, v_cache, pos, window, sinks, scale):
    """Shapes of both window calls (decode has no token axis)."""
    qs, ks, vs, dtype = q.shape, k.shape, v.shape, q.dtype
    rows = len(qs) == 4
    B, Hq, d, Hkv, dv = qs[0], qs[1], qs[-1], ks[1], vs[-1]
    N = qs[2] if rows else 1
    if not (-_INT < window < _INT and -_INT < sinks < _INT):
        raise ValueError(f"window and sinks must fit 32 bits, got {window} and {sinks}")
    if ks[0] != B or vs[0] != B or vs[1] != Hkv or ks[-1] != d or (rows and not ks[2] == vs[2] == N):
        raise ValueError(f"q, k, v do not fit: {list(qs)}, {list(ks)}, {list(vs)}")
    if out.shape != ((B, Hq, N, dv) if rows else (B, Hq, dv)):
        raise ValueError(f"out must be {[*qs[:-1], dv]}, got {list(out.shape)}")
    if not (k.dtype == dtype and v.dtype == dtype and out.dtype == dtype):
        raise ValueError("q, k, v and out must have one dtype")
    if k_cache is not None:
        _dense(k_cache, (B, Hkv, sinks + window, d), dtype, "k_cache")
    if v_cache is not None:
        _dense(v_cache, (B, Hkv, sinks + window, dv), dtype, "v_cache")
    if pos is not None:
        _dense(pos, (B,), _torch().int32, "pos")
    st = LaWindowStrides(*_head_strides(q, rows, "q"), *_head_strides(k, rows, "k"), *_head_strides(v, rows, "v"),
                         *_head_strides(out, rows, "out"))
    return B, Hq, Hkv, N, d, dv, float(d ** -0.5 if scale is None else scale), st


def la_window_prefill(q, k, v, window, sinks=0, k_cache=None, v_cache=None, pos=None, seq_lens=None, scale=None,
                      out=None, stream=None):
    """Sliding-window attention with sinks over prompts: q [B,Hq,N,d], k
    [B,Hkv,N,d], v [B,Hkv,N,dv] (bf16/fp32; batches, heads and rows may be
    strided).  With the rolling caches [B,Hkv,sinks+window,.] the tokens follow
    the pos[b] (int32, on the device; None: 0) cached ones and the caches are
    updated in place; pos itself is not.  seq_lens: host ints of a right-padded
    batch.  scale defaults to d ** -0.5.  Returns o [B,Hq,N,dv]."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B,Hq,N,d], k [B,Hkv,N,d] and v [B,Hkv,N,dv]")
    if out is None:
        out = _new((*q.shape[:-1], v.shape[-1]), q.dtype, q.device, stream)
    B, Hq, Hkv, N, d, dv, scale, st = _window_checks(q, k, v, out, k_cache, v_cache, pos, window, sinks, scale)
    cfg = LaConfig(_dtype_code(q), 0, 0.0, None, None, None, None, 0)
    cfg.stream, guard = _on_device(q, (k, v, out, k_cache, v_cache, pos), stream)
    with guard:
        rc = lib().la_window_prefill(_addr(q), _addr(k), _addr(v), _addr(out), _addr(k_cache), _addr(v_cache),
                                     _addr(pos), _lens_of(seq_lens, B), B, Hq, Hkv, N, d, dv, window, sinks,
                                     scale, ctypes.byref(st), ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_window_prefill")
    return out


def la_window_decode_step(q, k, v, k_cache, v_cache, pos, window, sinks=0, scale=None, out=None, stream=None):
    """One token of each sequence: q [B,Hq,d], k [B,Hkv,d], v [B,Hkv,dv] at
    position pos[b] (int32, on the device; negative: an idle sequence).  The
    caches take k and v in place.  Returns o [B,Hq,dv]."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q must be [B,Hq,d], k [B,Hkv,d] and v [B,Hkv,dv]")
    if out is None:
        out = _new((*q.shape[:-1], v.shape[-1]), q.dtype, q.device, stream)
    B, Hq, Hkv, N, d, dv, scale, st = _window_checks(q, k, v, out, k_cache, v_cache, pos, window, sinks, scale)
    cfg = LaConfig(_dtype_code(q), 0, 0.0, None, None, None, None, 0)
    cfg.stream, guard = _on_device(q, (k, v, out, k_cache, v_cache, pos), stream)
    with guard:
        rc = lib().la_window_decode_step(_addr(q), _addr(k), _addr(v), _addr(out), _addr(k_cache), _addr(v_cache),
                                         _addr(pos), B, Hq, Hkv, d, dv, window, sinks, scale, ctypes.byref(st),
                                         ctypes.byref(cfg))
    if rc != LA_OK:
        raise LaError(rc, "la_window_decode_step")
    return out


def la_set_stage_events(events=None):
    """Profiling hook: record torch.cuda.Event events[i] after the i-th kernel
    of every later call (None or [] turns it off).  The events must have been
    recorded once (so that they exist) and stay alive while the hook is set."""
    events = list(events or [])
    arr = (ctypes.c_void_p * max(1, len(events)))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    rc = lib().la_set_stage_events(arr, len(events))
    if rc != LA_OK:
        raise LaError(rc, "la_set_stage_events")


def la_selftest_wait_timeout(stream=None):
    """Enqueue the bounded-wait failure self-test; the next la_prefill_check
    on the stream raises LaError with code LA_ERR_TIMEOUT."""
    rc = lib().la_selftest_wait_timeout(_stream_handle(stream))
    if rc != LA_OK:
        raise LaError(rc, "la_selftest_wait_timeout")


def la_prefill_check(workspace=None, stream=None):
    """Synchronise the stream and report device-side errors of the last prefill."""
    rc = lib().la_prefill_check(_ptr(workspace), _stream_handle(stream))
    if rc != LA_OK:
        raise LaError(rc, "la_prefill_check")
