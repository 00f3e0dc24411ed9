"""Exact attention for one GB300 (sm_103a): Python binding of libfa.

The functions named like the C ABI (``fa_fwd``, ``fa_bwd``, ``fa_get_status``,
``fa_status_string``, ``fa_debug_set``, ``fa_debug_exp2``) only marshal
arguments: pointers may be given as ints or as CUDA tensors, the stream as an
int, a ``torch.cuda.Stream`` or None (the current stream). They return the
library's integer status. ``forward`` and ``backward`` allocate outputs with
torch, call the C ABI and raise ``FAError`` on a non-zero status.

Every computation runs in the CUDA kernels of libfa.so; there is no fallback.
If the library is missing the import of this module still succeeds (so it can
be built), but every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

__all__ = ["FAError", "lib", "fa_fwd", "fa_bwd", "fa_bwd_noalloc", "fa_bwd_launches", "fa_get_status", "fa_status_string", "fa_debug_set",
           "fa_debug_exp2", "fa_tune", "TUNE_EXP2_SPLIT", "TUNE_CTA_PAIRS", "TUNE_BWD_SPLIT", "fa_profile_events", "fa_trace", "forward", "backward", "STATUS",
           "fa_fwd_varlen", "fa_bwd_varlen", "fa_fwd_paged", "fa_cache_append", "forward_varlen", "backward_varlen",
           "forward_paged", "cache_append"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")

STATUS = {
    0: "FA_OK",
    1: "FA_ERR_INVALID_ARG",
    2: "FA_ERR_UNSUPPORTED",
    3: "FA_ERR_ALLOC",
    4: "FA_ERR_LAUNCH",
    5: "FA_ERR_TIMEOUT",
    6: "FA_ERR_NO_DEVICE",
}


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libfa.so (built in-tree). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfa.so is not built ({LIB_PATH}); run exact_attention_99_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, ull = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_ulonglong
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        L.fa_fwd.restype = i
        L.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
        L.fa_fwd_window.restype = i
        L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
        L.fa_fwd_fp8.restype = i
        L.fa_bwd.argtypes = [vp] * 9 + [i, i, i, i, i, i, f, i, vp]
        L.fa_step_host.argtypes = [vp] * 9 + [i, i, i, i, i, i, f, i, vp]
        L.fa_step_host.restype = i
        L.fa_bwd.restype = i
        L.fa_bwd_window.argtypes = [vp] * 9 + [i, i, i, i, i, i, f, i, i, vp]
        L.fa_bwd_window.restype = i
        L.fa_bwd_noalloc.argtypes = [vp] * 9 + [i, i, i, i, i, i, f, i, vp]
        L.fa_bwd_noalloc.restype = i
        L.fa_bwd_launches.argtypes = [i] * 7
        L.fa_bwd_launches.restype = i
        ll = ctypes.c_longlong
        L.fa_fwd_varlen.argtypes = [vp] * 7 + [i] * 6 + [ll, ll, ll, f, i, i, vp]
        L.fa_fwd_varlen.restype = i
        L.fa_bwd_varlen.argtypes = [vp] * 11 + [i] * 6 + [ll, ll, ll, f, i, i, vp]
        L.fa_bwd_varlen.restype = i
        L.fa_fwd_paged.argtypes = [vp] * 8 + [i] * 8 + [ll, f, i, i, vp]
        L.fa_fwd_paged.restype = i
        L.fa_cache_append.argtypes = [vp] * 7 + [i] * 7 + [ll, ll, vp]
        L.fa_cache_append.restype = i
        L.fa_get_status.argtypes = [vp]
        L.fa_get_status.restype = i
        L.fa_status_string.argtypes = [i]
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_debug_set.argtypes = [ull, i]
        L.fa_debug_set.restype = i
        L.fa_profile_events.argtypes = [vp, vp]
        L.fa_profile_events.restype = i
        L.fa_trace.argtypes = [vp]
        L.fa_trace.restype = i
        L.fa_debug_exp2.argtypes = [vp, vp, i, i, vp]
        L.fa_debug_exp2.restype = i
        L.fa_tune.argtypes = [i, i]
        L.fa_tune.restype = i
        _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def fa_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=None) -> int:
    return lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, float(scale),
                        int(causal), _stream(stream))


def fa_fwd_window(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, window_left, window_right, stream=None) -> int:
    return lib().fa_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, float(scale),
                               int(window_left), int(window_right), _stream(stream))


def fa_step_host(q, k, v, dout, o, lse, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=None) -> int:
    """Forward + backward on host (CPU, preferably pinned) tensors; see fa.h fa_step_host."""
    return lib().fa_step_host(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(o), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                              B, Hq, Hkv, Nq, Nk, d, float(scale), int(causal), _stream(stream))


def fa_fwd_fp8(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, incoherent=1, stream=None) -> int:
    return lib().fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, float(scale),
                            int(causal), int(incoherent), _stream(stream))


def forward_fp8(q, k, v, causal: bool = False, scale: float | None = None, incoherent: bool = True, stream=None):
    """O, LSE of the e4m3 forward (d = 128; see fa.h fa_fwd_fp8)."""
    import torch
    B, Nq, Hq, d = q.shape
    _, Nk, Hkv, _ = k.shape
    _check_bshd("q", q, B, Nq, Hq, d)
    _check_bshd("k", k, B, Nk, Hkv, d)
    _check_bshd("v", v, B, Nk, Hkv, d)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    st = fa_fwd_fp8(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, int(incoherent), stream)
    if st != 0:
        raise FAError(st, "fa_fwd_fp8")
    return o, lse


def _window_args(causal, window):
    """(left, right) bounds for the *_window calls; causal caps right at 0."""
    wl, wr = (-1, -1) if window is None else (int(window[0]), int(window[1]))
    if causal:
        wr = 0 if wr < 0 else min(wr, 0)
    return wl, wr


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=None) -> int:
    return lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                        B, Hq, Hkv, Nq, Nk, d, float(scale), int(causal), _stream(stream))


def fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, window_left, window_right,
                  stream=None) -> int:
    return lib().fa_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                               _ptr(dv), B, Hq, Hkv, Nq, Nk, d, float(scale), int(window_left), int(window_right),
                               _stream(stream))


def fa_bwd_launches(B, Hq, Hkv, Nq, Nk, d, causal) -> int:
    """Kernels fa_bwd launches for this problem (see fa.h), or minus a status."""
    return lib().fa_bwd_launches(int(B), int(Hq), int(Hkv), int(Nq), int(Nk), int(d), int(causal))


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream=None) -> int:
    """fa_bwd with its workspace in the library's fixed device array (no
    device allocation during the call; see fa.h for the size limit)."""
    return lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                _ptr(dv), B, Hq, Hkv, Nq, Nk, d, float(scale), int(causal), _stream(stream))


def fa_get_status(stream=None) -> int:
    return lib().fa_get_status(_stream(stream))


def fa_status_string(status: int) -> str:
    return lib().fa_status_string(int(status)).decode()


def fa_debug_set(wait_limit_ns: int = 0, inject: int = 0) -> int:
    return lib().fa_debug_set(int(wait_limit_ns), int(inject))


def fa_profile_events(begin=None, end=None) -> int:
    """begin/end: torch.cuda.Event (created with enable_timing) or None."""
    b = None if begin is None else begin.cuda_event
    e = None if end is None else end.cuda_event
    return lib().fa_profile_events(b, e)


TRACE_CTAS, TRACE_STEPS, TRACE_POINTS = 4, 64, 16


def fa_trace(buf=None) -> int:
    """buf: CUDA int64 tensor of TRACE_CTAS*TRACE_STEPS*TRACE_POINTS words, or None."""
    return lib().fa_trace(_ptr(buf))


TUNE_EXP2_SPLIT = 1
TUNE_CTA_PAIRS = 2
TUNE_BWD_SPLIT = 3


def fa_tune(knob: int, value: int) -> int:
    """Process-wide tuning knob (see fa.h fa_tune); TUNE_EXP2_SPLIT: 0 = every
    forward exponential on the special-function unit, N in {1, 2, 4, 8} = one
    column pair in every N on the FMA-pipe polynomial; TUNE_CTA_PAIRS: 1 = the
    d = 128 forward on pairs of CTAs (cta_group::2), 0 = one CTA per SM;
    TUNE_BWD_SPLIT: -1 = the causal backward's split count from its model,
    m >= 0 = that many pairs per kv head run as single tiles."""
    return lib().fa_tune(int(knob), int(value))


def fa_debug_exp2(x, y, n, mode, stream=None) -> int:
    return lib().fa_debug_exp2(_ptr(x), _ptr(y), int(n), int(mode), _stream(stream))


def _check_bshd(name, t, B, N, H, d):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (B, N, H, d):
        raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor of shape {(B, N, H, d)}")


def forward(q, k, v, causal: bool = False, scale: float | None = None, out=None, stream=None, window=None):
    """O, LSE for q [B,Nq,Hq,d], k/v [B,Nk,Hkv,d] (bf16, CUDA, contiguous).
    window: optional (left, right) sliding-window bounds (see fa.h)."""
    import torch
    B, Nq, Hq, d = q.shape
    _, Nk, Hkv, _ = k.shape
    _check_bshd("q", q, B, Nq, Hq, d)
    _check_bshd("k", k, B, Nk, Hkv, d)
    _check_bshd("v", v, B, Nk, Hkv, d)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    else:
        o, lse = out
    if window is None:
        st = fa_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream)
    else:
        st = fa_fwd_window(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, *_window_args(causal, window), stream)
    if st != 0:
        raise FAError(st, "fa_fwd")
    return o, lse


def backward(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, out=None, stream=None,
             window=None):
    """dQ, dK, dV for the forward that produced o and lse (same causal flag
    and window)."""
    import torch
    B, Nq, Hq, d = q.shape
    _, Nk, Hkv, _ = k.shape
    for name, t, N, H in (("q", q, Nq, Hq), ("k", k, Nk, Hkv), ("v", v, Nk, Hkv), ("o", o, Nq, Hq),
                          ("dout", dout, Nq, Hq)):
        _check_bshd(name, t, B, N, H, d)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    else:
        dq, dk, dv = out
    if window is None:
        st = fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, causal, stream)
    else:
        st = fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale,
                           *_window_args(causal, window), stream)
    if st != 0:
        raise FAError(st, "fa_bwd")
    return dq, dk, dv


# --- sequences of different lengths (see fa.h) ---------------------------------

def fa_fwd_varlen(q, k, v, o, lse, cu_q, cu_k, B, Hq, Hkv, total_q, total_k, d, q_stride, k_stride, v_stride, scale,
                  window_left, window_right, stream=None) -> int:
    return lib().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_q), _ptr(cu_k), B, Hq, Hkv,
                               total_q, total_k, d, q_stride, k_stride, v_stride, float(scale), int(window_left),
                               int(window_right), _stream(stream))


def fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, B, Hq, Hkv, total_q, total_k, d, q_stride, k_stride,
                  v_stride, scale, window_left, window_right, stream=None) -> int:
    return lib().fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                               _ptr(cu_q), _ptr(cu_k), B, Hq, Hkv, total_q, total_k, d, q_stride, k_stride, v_stride,
                               float(scale), int(window_left), int(window_right), _stream(stream))


def fa_fwd_paged(q, k_pages, v_pages, o, lse, cu_q, lens_k, page_table, B, Hq, Hkv, total_q, num_pages, page_size,
                 max_pages, d, q_stride, scale, window_left, window_right, stream=None) -> int:
    return lib().fa_fwd_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(o), _ptr(lse), _ptr(cu_q), _ptr(lens_k),
                              _ptr(page_table), B, Hq, Hkv, total_q, num_pages, page_size, max_pages, d, q_stride,
                              float(scale), int(window_left), int(window_right), _stream(stream))


def fa_cache_append(k, v, k_pages, v_pages, cu_q, lens_k, page_table, B, Hkv, total_q, num_pages, page_size, max_pages,
                    d, k_stride, v_stride, stream=None) -> int:
    return lib().fa_cache_append(_ptr(k), _ptr(v), _ptr(k_pages), _ptr(v_pages), _ptr(cu_q), _ptr(lens_k),
                                 _ptr(page_table), B, Hkv, total_q, num_pages, page_size, max_pages, d, k_stride,
                                 v_stride, _stream(stream))


def _tokens(name, t, device=None, shape=None):
    """Checks a packed [total, H, d] tensor; returns its elements between tokens."""
    import torch
    if t.dim() != 3 or t.dtype != torch.bfloat16 or not t.is_cuda or t.shape[1] < 1:
        raise ValueError(f"{name} must be a CUDA bf16 tensor of shape [tokens, heads, d]")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, q is on {device}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have the shape {shape}")
    n, h, d = t.shape
    s = t.stride()
    if n <= 1:  # the stride of an axis of one has no meaning
        s = (h * d, s[1], s[2])
    if s[2] != 1 or (h > 1 and s[1] != d) or s[0] < h * d:
        raise ValueError(f"{name}: the heads of a token must be contiguous, and tokens must not overlap")
    return s[0]


def _ints(name, t, shape, device):
    import torch
    if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape} on {device}")


def _pages(k_pages, v_pages, hkv, d, device):
    import torch
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if (t.dtype != torch.bfloat16 or t.dim() != 4 or t.shape != k_pages.shape or tuple(t.shape[2:]) != (hkv, d)
                or not t.is_contiguous() or t.device != device):
            raise ValueError(f"{name} must be a contiguous bf16 tensor of shape [pages, page_size, {hkv}, {d}] on {device}")
    return k_pages.shape[0], k_pages.shape[1]


class _on:
    """The device of the call's tensors made current, and the call's stream
    for the outputs that it allocates (so that the allocator reuses their
    memory in that stream's order)."""

    def __init__(self, device, stream):
        import torch
        self.guards = []
        if device.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(device))
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=device)
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _packed(name, t, shape, device):
    import torch
    if tuple(t.shape) != shape or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous bf16 tensor of shape {shape} on {device}")


def _seq_out(q, out):
    """The given (o, lse) after a check, or new ones."""
    import torch
    total, hq, d = q.shape
    if out is None:
        return (torch.empty((total, hq, d), device=q.device, dtype=torch.bfloat16),
                torch.empty((hq, total), device=q.device, dtype=torch.float32))
    o, lse = out
    _packed("o", o, (total, hq, d), q.device)
    if tuple(lse.shape) != (hq, total) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != q.device:
        raise ValueError(f"lse must be a contiguous fp32 tensor of shape {(hq, total)} on {q.device}")
    return o, lse


def forward_varlen(q, k, v, cu_q, cu_k, causal: bool = False, scale: float | None = None, out=None, stream=None,
                   window=None):
    """O [total_q, Hq, d] and LSE [Hq, total_q] of packed sequences: q
    [total_q, Hq, d], k/v [total_k, Hkv, d] (bf16, CUDA; tokens may be strided),
    cu_q, cu_k int32 [B + 1] row offsets on the device (see fa.h fa_fwd_varlen).
    Rows outside every sequence are left as they are (unset in new outputs)."""
    qs = _tokens("q", q)
    total_q, hq, d = q.shape
    total_k, hkv = k.shape[0], k.shape[1]
    ks, vs = _tokens("k", k, q.device, (total_k, hkv, d)), _tokens("v", v, q.device, (total_k, hkv, d))
    B = cu_q.shape[0] - 1
    _ints("cu_q", cu_q, (B + 1,), q.device)
    _ints("cu_k", cu_k, (B + 1,), q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    with _on(q.device, stream):
        o, lse = _seq_out(q, out)
        st = fa_fwd_varlen(q, k, v, o, lse, cu_q, cu_k, B, hq, hkv, total_q, total_k, d, qs, ks, vs, scale,
                           *_window_args(causal, window))
    if st != 0:
        raise FAError(st, "fa_fwd_varlen")
    return o, lse


def backward_varlen(q, k, v, o, lse, dout, cu_q, cu_k, causal: bool = False, scale: float | None = None, out=None,
                    stream=None, window=None):
    """dQ [total_q, Hq, d], dK, dV [total_k, Hkv, d] for the forward_varlen
    that gave o and lse (same offsets, mask and scale); dout [total_q, Hq, d].
    Rows outside every sequence are left as they are (unset in new outputs)."""
    import torch
    qs = _tokens("q", q)
    total_q, hq, d = q.shape
    total_k, hkv = k.shape[0], k.shape[1]
    ks, vs = _tokens("k", k, q.device, (total_k, hkv, d)), _tokens("v", v, q.device, (total_k, hkv, d))
    B = cu_q.shape[0] - 1
    _ints("cu_q", cu_q, (B + 1,), q.device)
    _ints("cu_k", cu_k, (B + 1,), q.device)
    _seq_out(q, (o, lse))
    _packed("dout", dout, (total_q, hq, d), q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    with _on(q.device, stream):
        if out is None:
            dq, dk, dv = (torch.empty(s, device=q.device, dtype=torch.bfloat16)
                          for s in ((total_q, hq, d), (total_k, hkv, d), (total_k, hkv, d)))
        else:
            dq, dk, dv = out
            _packed("dq", dq, (total_q, hq, d), q.device)
            _packed("dk", dk, (total_k, hkv, d), q.device)
            _packed("dv", dv, (total_k, hkv, d), q.device)
        st = fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, B, hq, hkv, total_q, total_k, d, qs, ks, vs,
                           scale, *_window_args(causal, window))
    if st != 0:
        raise FAError(st, "fa_bwd_varlen")
    return dq, dk, dv


def forward_paged(q, k_pages, v_pages, cu_q, lens_k, page_table, causal: bool = True, scale: float | None = None,
                  out=None, stream=None, window=None):
    """O [total_q, Hq, d] and LSE [Hq, total_q] of new tokens q [total_q, Hq, d]
    (bf16, CUDA; tokens may be strided) over a cache of pages [num_pages,
    page_size, Hkv, d]; cu_q [B + 1], lens_k [B] and page_table [B, max_pages]
    are int32 on the device (see fa.h fa_fwd_paged)."""
    qs = _tokens("q", q)
    total_q, hq, d = q.shape
    hkv = k_pages.shape[2] if k_pages.dim() == 4 else 0
    num_pages, page_size = _pages(k_pages, v_pages, hkv, d, q.device)
    B = cu_q.shape[0] - 1
    max_pages = page_table.shape[-1]
    _ints("cu_q", cu_q, (B + 1,), q.device)
    _ints("lens_k", lens_k, (B,), q.device)
    _ints("page_table", page_table, (B, max_pages), q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    with _on(q.device, stream):
        o, lse = _seq_out(q, out)
        st = fa_fwd_paged(q, k_pages, v_pages, o, lse, cu_q, lens_k, page_table, B, hq, hkv, total_q, num_pages,
                          page_size, max_pages, d, qs, scale, *_window_args(causal, window))
    if st != 0:
        raise FAError(st, "fa_fwd_paged")
    return o, lse


def cache_append(k, v, k_pages, v_pages, cu_q, lens_k, page_table, stream=None) -> None:
    """k, v [total_q, Hkv, d] of new tokens (bf16, CUDA; tokens may be strided)
    into the pages, in place; lens_k are the lengths with the new tokens (see
    fa.h fa_cache_append)."""
    ks = _tokens("k", k)
    total, hkv, d = k.shape
    vs = _tokens("v", v, k.device, (total, hkv, d))
    num_pages, page_size = _pages(k_pages, v_pages, hkv, d, k.device)
    B = cu_q.shape[0] - 1
    max_pages = page_table.shape[-1]
    _ints("cu_q", cu_q, (B + 1,), k.device)
    _ints("lens_k", lens_k, (B,), k.device)
    _ints("page_table", page_table, (B, max_pages), k.device)
    with _on(k.device, stream):
        st = fa_cache_append(k, v, k_pages, v_pages, cu_q, lens_k, page_table, B, hkv, total, num_pages, page_size,
                             max_pages, d, ks, vs)
    if st != 0:
        raise FAError(st, "fa_cache_append")
