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
           "forward_paged", "cache_append", "fa_fwd_paged_fp8", "fa_cache_append_fp8", "fa_rotary", "forward_paged_fp8",
           "cache_append_fp8", "rotary", "rotary_backward", "rotary_frequencies"]

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
        L.fa_fwd_paged_fp8.argtypes = [vp] * 10 + [i] * 8 + [ll, f, i, i, vp]
        L.fa_fwd_paged_fp8.restype = i
        L.fa_cache_append_fp8.argtypes = [vp] * 9 + [i] * 7 + [ll, ll, vp]
        L.fa_cache_append_fp8.restype = i
        L.fa_rotary.argtypes = [vp] * 7 + [i] * 6 + [ll] * 4 + [f, i, i, vp]
        L.fa_rotary.restype = i
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


_raw_stream = _get_device = None


def _current_stream() -> int:
    """The current stream's handle (without building a Stream object, which
    takes longer than a small call's checks)."""
    global _raw_stream, _get_device
    if _raw_stream is None:
        import torch
        torch.cuda.init()
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _raw_stream(_get_device())


def _stream(s):
    if s is None:
        return _current_stream()
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
    # (C ints: a bound past 31 bits is past every length, any negative one is no limit)
    wl, wr = (-1, -1) if window is None else (max(-1, min(int(w), 2 ** 31 - 1)) for w in window)
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


def fa_fwd_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, o, lse, cu_q, lens_k, page_table, B, Hq, Hkv, total_q,
                     num_pages, page_size, max_pages, d, q_stride, scale, window_left, window_right, stream=None) -> int:
    return lib().fa_fwd_paged_fp8(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales), _ptr(o),
                                  _ptr(lse), _ptr(cu_q), _ptr(lens_k), _ptr(page_table), B, Hq, Hkv, total_q, num_pages,
                                  page_size, max_pages, d, q_stride, float(scale), int(window_left), int(window_right),
                                  _stream(stream))


def fa_cache_append_fp8(k, v, k_pages, v_pages, k_scales, v_scales, cu_q, lens_k, page_table, B, Hkv, total_q, num_pages,
                        page_size, max_pages, d, k_stride, v_stride, stream=None) -> int:
    return lib().fa_cache_append_fp8(_ptr(k), _ptr(v), _ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales),
                                     _ptr(cu_q), _ptr(lens_k), _ptr(page_table), B, Hkv, total_q, num_pages, page_size,
                                     max_pages, d, k_stride, v_stride, _stream(stream))


def fa_rotary(q, k, q_out, k_out, inv_freq, cu_q, lens, B, Hq, Hk, total, d, rot, q_stride, k_stride, q_out_stride,
              k_out_stride, mscale, interleaved, transposed, stream=None) -> int:
    return lib().fa_rotary(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr(inv_freq), _ptr(cu_q), _ptr(lens), B, Hq, Hk,
                           total, d, rot, q_stride, k_stride, q_out_stride, k_out_stride, float(mscale), int(interleaved),
                           int(transposed), _stream(stream))


_bf16 = _i32 = _f32 = _e4m3 = _empty = None


def _types():
    global _bf16, _i32, _f32, _e4m3, _empty
    import torch
    _bf16, _i32, _f32, _e4m3, _empty = torch.bfloat16, torch.int32, torch.float32, torch.float8_e4m3fn, torch.empty


def _tokens(name, t, device, shape):
    """Checks a packed [total, H, d] tensor; returns its elements between tokens."""
    if t.dtype != _bf16 or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name} must be a bf16 tensor of shape {tuple(shape)} on cuda:{device}")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if n <= 1:  # the stride of an axis of one has no meaning
        s0 = h * d
    if s2 != 1 or (s1 != d and h > 1) or s0 < h * d:
        raise ValueError(f"{name}: the heads of a token must be contiguous, and tokens must not overlap")
    return s0


def _first(name, t):
    """The device index of a call's first tensor, after a check of its form."""
    if _bf16 is None:
        _types()
    if t.dim() != 3 or not t.is_cuda or t.shape[1] < 1:
        raise ValueError(f"{name} must be a CUDA bf16 tensor of shape [tokens, heads, d]")
    return t.get_device()


def _ints(name, t, shape, device):
    if t.dtype != _i32 or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on cuda:{device}")


def _packed(name, t, shape, device, dtype=None):
    if t.shape != shape or t.dtype != (dtype or _bf16) or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a contiguous {dtype or _bf16} tensor of shape {tuple(shape)} on cuda:{device}")


def _pages(k_pages, v_pages, hkv, d, device, dtype=None):
    shape = k_pages.shape
    if len(shape) != 4 or shape[2] != hkv or shape[3] != d:
        raise ValueError(f"k_pages must have the shape [pages, page_size, {hkv}, {d}]")
    _packed("k_pages", k_pages, shape, device, dtype)
    _packed("v_pages", v_pages, shape, device, dtype)
    return shape[0], shape[1]


class _on:
    """The device of the call's tensors made current, and the call's stream
    for the outputs that it allocates (so that the allocator reuses their
    memory in that stream's order)."""

    def __init__(self, device, stream):
        import torch
        self.guards = []
        if device != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(device))
        if stream is not None:
            if isinstance(stream, int):
                # (0 is the default stream's handle, and ExternalStream(0) some new stream)
                stream = (torch.cuda.ExternalStream(stream, device=torch.device("cuda", device)) if stream != 0
                          else torch.cuda.default_stream(device))
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _here(device, stream):
    """The current stream's handle if the call may be made as things are: its
    tensors on the current device and no other stream asked for. Else None."""
    if _raw_stream is None:
        _current_stream()
    return _raw_stream(device) if stream is None and device == _get_device() else None


def _seq_out(q, shape, out):
    """The given (o, lse) after a check, or new ones."""
    total, hq, _ = shape
    if out is None:
        return _empty(shape, dtype=_bf16, device=q.device), _empty((hq, total), dtype=_f32, device=q.device)
    o, lse = out
    _packed("o", o, shape, q.get_device())
    _packed("lse", lse, (hq, total), q.get_device(), _f32)
    return o, lse


def _fwd_varlen(stream, q, k, v, cu_q, cu_k, out, shape, kshape, strides, scale, wl, wr):
    o, lse = _seq_out(q, shape, out)
    total_q, hq, d = shape
    total_k, hkv, _ = kshape
    st = lib().fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), cu_q.data_ptr(),
                             cu_k.data_ptr(), cu_q.shape[0] - 1, hq, hkv, total_q, total_k, d, *strides, scale, wl, wr,
                             stream)
    if st != 0:
        raise FAError(st, "fa_fwd_varlen")
    return o, lse


def _varlen_args(q, k, v, cu_q, cu_k):
    """Checks shared by forward_varlen and backward_varlen: device, shapes, token strides."""
    device = _first("q", q)
    shape, kshape = q.shape, k.shape
    if len(kshape) != 3 or kshape[2] != shape[2] or kshape[1] < 1:
        raise ValueError(f"k must have the shape [tokens, kv heads, {shape[2]}]")
    strides = _tokens("q", q, device, shape), _tokens("k", k, device, kshape), _tokens("v", v, device, kshape)
    n = cu_q.shape
    _ints("cu_q", cu_q, n, device)
    if cu_k is not cu_q:
        _ints("cu_k", cu_k, n, device)
    if len(n) != 1 or n[0] < 2:
        raise ValueError("cu_q must hold the row offsets of one sequence at least")
    return device, shape, kshape, strides


def forward_varlen(q, k, v, cu_q, cu_k, causal: bool = False, scale: float | None = None, out=None, stream=None,
                   window=None):
    """O [total_q, Hq, d] and LSE [Hq, total_q] of packed sequences: q
    [total_q, Hq, d], k/v [total_k, Hkv, d] (bf16, CUDA; tokens may be strided),
    cu_q, cu_k int32 [B + 1] row offsets on the device (see fa.h fa_fwd_varlen).
    Rows outside every sequence are left as they are (unset in new outputs)."""
    device, shape, kshape, strides = _varlen_args(q, k, v, cu_q, cu_k)
    scale = 1.0 / math.sqrt(shape[2]) if scale is None else scale
    wl, wr = (-1, 0 if causal else -1) if window is None else _window_args(causal, window)
    s = _here(device, stream)
    if s is not None:
        return _fwd_varlen(s, q, k, v, cu_q, cu_k, out, shape, kshape, strides, scale, wl, wr)
    with _on(device, stream):
        return _fwd_varlen(_current_stream(), q, k, v, cu_q, cu_k, out, shape, kshape, strides, scale, wl, wr)


def _bwd_varlen(stream, q, k, v, o, lse, dout, cu_q, cu_k, out, shape, kshape, strides, scale, wl, wr):
    total_q, hq, d = shape
    total_k, hkv, _ = kshape
    if out is None:
        dq, dk, dv = (_empty(x, dtype=_bf16, device=q.device) for x in (shape, kshape, kshape))
    else:
        dq, dk, dv = out
        device = q.get_device()
        _packed("dq", dq, shape, device)
        _packed("dk", dk, kshape, device)
        _packed("dv", dv, kshape, device)
    st = lib().fa_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
                             cu_q.shape[0] - 1, hq, hkv, total_q, total_k, d, *strides, scale, wl, wr, stream)
    if st != 0:
        raise FAError(st, "fa_bwd_varlen")
    return dq, dk, dv


def backward_varlen(q, k, v, o, lse, dout, cu_q, cu_k, causal: bool = False, scale: float | None = None, out=None,
                    stream=None, window=None):
    """dQ [total_q, Hq, d], dK, dV [total_k, Hkv, d] for the forward_varlen
    that gave o and lse (same offsets, mask and scale); dout [total_q, Hq, d].
    Rows outside every sequence are left as they are (unset in new outputs)."""
    device, shape, kshape, strides = _varlen_args(q, k, v, cu_q, cu_k)
    _seq_out(q, shape, (o, lse))
    _packed("dout", dout, shape, device)
    scale = 1.0 / math.sqrt(shape[2]) if scale is None else scale
    wl, wr = (-1, 0 if causal else -1) if window is None else _window_args(causal, window)
    s = _here(device, stream)
    if s is not None:
        return _bwd_varlen(s, q, k, v, o, lse, dout, cu_q, cu_k, out, shape, kshape, strides, scale, wl, wr)
    with _on(device, stream):
        return _bwd_varlen(_current_stream(), q, k, v, o, lse, dout, cu_q, cu_k, out, shape, kshape, strides, scale, wl, wr)


def _cache_args(k_pages, v_pages, cu_q, lens_k, page_table, hkv, d, device, dtype=None):
    """Checks shared by the calls over a paged cache: B, pages, page size, pages of a sequence."""
    num_pages, page_size = _pages(k_pages, v_pages, hkv, d, device, dtype)
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must have the shape [sequences, pages]")
    B, max_pages = shape
    _ints("cu_q", cu_q, (B + 1,), device)
    _ints("lens_k", lens_k, (B,), device)
    _ints("page_table", page_table, shape, device)
    return B, num_pages, page_size, max_pages


def _fwd_paged(stream, q, k_pages, v_pages, cu_q, lens_k, page_table, out, shape, qs, hkv, sizes, scale, wl, wr):
    o, lse = _seq_out(q, shape, out)
    total_q, hq, d = shape
    B, num_pages, page_size, max_pages = sizes
    st = lib().fa_fwd_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), o.data_ptr(), lse.data_ptr(),
                            cu_q.data_ptr(), lens_k.data_ptr(), page_table.data_ptr(), B, hq, hkv, total_q, num_pages,
                            page_size, max_pages, d, qs, scale, wl, wr, stream)
    if st != 0:
        raise FAError(st, "fa_fwd_paged")
    return o, lse


def forward_paged(q, k_pages, v_pages, cu_q, lens_k, page_table, causal: bool = True, scale: float | None = None,
                  out=None, stream=None, window=None):
    """O [total_q, Hq, d] and LSE [Hq, total_q] of new tokens q [total_q, Hq, d]
    (bf16, CUDA; tokens may be strided) over a cache of pages [num_pages,
    page_size, Hkv, d]; cu_q [B + 1], lens_k [B] and page_table [B, max_pages]
    are int32 on the device (see fa.h fa_fwd_paged)."""
    device = _first("q", q)
    shape = q.shape
    qs = _tokens("q", q, device, shape)
    hkv = k_pages.shape[2] if k_pages.dim() == 4 else 0
    sizes = _cache_args(k_pages, v_pages, cu_q, lens_k, page_table, hkv, shape[2], device)
    scale = 1.0 / math.sqrt(shape[2]) if scale is None else scale
    wl, wr = (-1, 0 if causal else -1) if window is None else _window_args(causal, window)
    s = _here(device, stream)
    if s is not None:
        return _fwd_paged(s, q, k_pages, v_pages, cu_q, lens_k, page_table, out, shape, qs, hkv, sizes, scale, wl, wr)
    with _on(device, stream):
        return _fwd_paged(_current_stream(), q, k_pages, v_pages, cu_q, lens_k, page_table, out, shape, qs, hkv, sizes,
                          scale, wl, wr)


def _append(stream, k, v, k_pages, v_pages, cu_q, lens_k, page_table, shape, ks, vs, sizes):
    total, hkv, d = shape
    B, num_pages, page_size, max_pages = sizes
    st = lib().fa_cache_append(k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), cu_q.data_ptr(),
                               lens_k.data_ptr(), page_table.data_ptr(), B, hkv, total, num_pages, page_size, max_pages,
                               d, ks, vs, stream)
    if st != 0:
        raise FAError(st, "fa_cache_append")


def cache_append(k, v, k_pages, v_pages, cu_q, lens_k, page_table, stream=None) -> None:
    """k, v [total_q, Hkv, d] of new tokens (bf16, CUDA; tokens may be strided)
    into the pages, in place; lens_k are the lengths with the new tokens (see
    fa.h fa_cache_append)."""
    device = _first("k", k)
    shape = k.shape
    ks, vs = _tokens("k", k, device, shape), _tokens("v", v, device, shape)
    sizes = _cache_args(k_pages, v_pages, cu_q, lens_k, page_table, shape[1], shape[2], device)
    s = _here(device, stream)
    if s is not None:
        return _append(s, k, v, k_pages, v_pages, cu_q, lens_k, page_table, shape, ks, vs, sizes)
    with _on(device, stream):
        _append(_current_stream(), k, v, k_pages, v_pages, cu_q, lens_k, page_table, shape, ks, vs, sizes)


# --- a cache in 8 bits (see fa.h) -----------------------------------------------

def _cache8_args(k_pages, v_pages, k_scales, v_scales, cu_q, lens_k, page_table, hkv, d, device):
    """_cache_args of an e4m3 cache, with its scales."""
    shape, table = k_pages.shape, page_table.shape
    if len(shape) == 4 and len(table) == 2:
        num_pages, page_size, h, dd = shape
        B, max_pages = table
        # all in one expression, the small calls' time; what is wrong is said below
        if (h == hkv and dd == d and k_pages.dtype is _e4m3 and v_pages.dtype is _e4m3 and v_pages.shape == shape
                and k_scales.dtype is _f32 and v_scales.dtype is _f32
                and k_scales.shape == (num_pages, page_size // 16, hkv) and v_scales.shape == k_scales.shape
                and cu_q.dtype is _i32 and lens_k.dtype is _i32 and page_table.dtype is _i32
                and cu_q.shape == (B + 1,) and lens_k.shape == (B,)
                and k_pages.is_contiguous() and v_pages.is_contiguous() and k_scales.is_contiguous()
                and v_scales.is_contiguous() and cu_q.is_contiguous() and lens_k.is_contiguous()
                and page_table.is_contiguous()
                and k_pages.get_device() == v_pages.get_device() == k_scales.get_device() == v_scales.get_device()
                == cu_q.get_device() == lens_k.get_device() == page_table.get_device() == device):
            return B, num_pages, page_size, max_pages
    sizes = _cache_args(k_pages, v_pages, cu_q, lens_k, page_table, hkv, d, device, _e4m3)
    shape = (sizes[1], sizes[2] // 16, hkv)
    _packed("k_scales", k_scales, shape, device, _f32)
    _packed("v_scales", v_scales, shape, device, _f32)
    return sizes


def _fwd_paged8(stream, q, pages, cu_q, lens_k, page_table, out, shape, qs, hkv, sizes, scale, wl, wr):
    o, lse = _seq_out(q, shape, out)
    total_q, hq, d = shape
    B, num_pages, page_size, max_pages = sizes
    st = lib().fa_fwd_paged_fp8(q.data_ptr(), *(x.data_ptr() for x in pages), o.data_ptr(), lse.data_ptr(),
                                cu_q.data_ptr(), lens_k.data_ptr(), page_table.data_ptr(), B, hq, hkv, total_q,
                                num_pages, page_size, max_pages, d, qs, scale, wl, wr, stream)
    if st != 0:
        raise FAError(st, "fa_fwd_paged_fp8")
    return o, lse


def forward_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, cu_q, lens_k, page_table, causal: bool = True,
                      scale: float | None = None, out=None, stream=None, window=None):
    """forward_paged over a cache in 8 bits: pages [num_pages, page_size, Hkv, d]
    of torch.float8_e4m3fn, scales [num_pages, page_size / 16, Hkv] fp32 (see fa.h
    fa_fwd_paged_fp8)."""
    device = _first("q", q)
    shape = q.shape
    qs = _tokens("q", q, device, shape)
    hkv = k_pages.shape[2] if k_pages.dim() == 4 else 0
    sizes = _cache8_args(k_pages, v_pages, k_scales, v_scales, cu_q, lens_k, page_table, hkv, shape[2], device)
    scale = 1.0 / math.sqrt(shape[2]) if scale is None else scale
    wl, wr = (-1, 0 if causal else -1) if window is None else _window_args(causal, window)
    pages = (k_pages, v_pages, k_scales, v_scales)
    s = _here(device, stream)
    if s is not None:
        return _fwd_paged8(s, q, pages, cu_q, lens_k, page_table, out, shape, qs, hkv, sizes, scale, wl, wr)
    with _on(device, stream):
        return _fwd_paged8(_current_stream(), q, pages, cu_q, lens_k, page_table, out, shape, qs, hkv, sizes, scale, wl, wr)


def _append8(stream, k, v, pages, cu_q, lens_k, page_table, shape, ks, vs, sizes):
    total, hkv, d = shape
    B, num_pages, page_size, max_pages = sizes
    st = lib().fa_cache_append_fp8(k.data_ptr(), v.data_ptr(), *(x.data_ptr() for x in pages), cu_q.data_ptr(),
                                   lens_k.data_ptr(), page_table.data_ptr(), B, hkv, total, num_pages, page_size,
                                   max_pages, d, ks, vs, stream)
    if st != 0:
        raise FAError(st, "fa_cache_append_fp8")


def cache_append_fp8(k, v, k_pages, v_pages, k_scales, v_scales, cu_q, lens_k, page_table, stream=None) -> None:
    """k, v [total_q, Hkv, d] of new tokens (bf16, CUDA; tokens may be strided)
    into the pages of a cache in 8 bits, in place, with a scale for each block
    of 16 tokens and head (see fa.h fa_cache_append_fp8)."""
    device = _first("k", k)
    shape = k.shape
    ks, vs = _tokens("k", k, device, shape), _tokens("v", v, device, shape)
    sizes = _cache8_args(k_pages, v_pages, k_scales, v_scales, cu_q, lens_k, page_table, shape[1], shape[2], device)
    pages = (k_pages, v_pages, k_scales, v_scales)
    s = _here(device, stream)
    if s is not None:
        return _append8(s, k, v, pages, cu_q, lens_k, page_table, shape, ks, vs, sizes)
    with _on(device, stream):
        _append8(_current_stream(), k, v, pages, cu_q, lens_k, page_table, shape, ks, vs, sizes)


# --- rotary positions (see fa.h) --------------------------------------------------

def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq, mscale) for `rotary`: dim / 2 inverse frequencies (fp32, on
    the CPU) and the factor of the turned values, computed in 64 bits.

    f_j = base^(-2 j / dim). `scaling`, for contexts `factor` times as long as
    those that a model was made for:
      None       f_j;
      "linear"   f_j / factor: all places are drawn together;
      "ntk"      the base times factor^(dim / (dim - 2)): the slowest pair turns
                 by 1 / factor, the fastest as before;
      "yarn"     between f_j and f_j / factor by how often the pair turns within
                 original_length places: f_j from beta_fast turns on, f_j /
                 factor up to beta_slow, a line over j between; mscale is
                 0.1 ln(factor) + 1.
    """
    import torch
    if dim < 2 or dim % 2 or not base > 1.0 or not math.isfinite(base):
        raise ValueError("rotary_frequencies: dim must be even and base finite and above 1")
    if not (math.isfinite(factor) and factor >= 1.0):
        raise ValueError("rotary_frequencies: factor must be finite and 1 at least")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"rotary_frequencies: no scaling {scaling!r}")
    mscale = 1.0
    if scaling == "ntk" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = [base ** (-2.0 * j / dim) for j in range(dim // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "yarn":
        if original_length is None or original_length < 1 or not beta_fast > beta_slow > 0:
            raise ValueError("rotary_frequencies: yarn needs original_length and beta_fast > beta_slow > 0")

        def pair_of(turns):  # the (fractional) pair that turns so often within original_length
            return dim * math.log(original_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        lo = max(math.floor(pair_of(beta_fast)), 0)
        hi = min(math.ceil(pair_of(beta_slow)), dim - 1)
        span = max(hi - lo, 0.001)
        f = [x / factor * r + x * (1.0 - r) for j, x in enumerate(f) for r in (min(max((j - lo) / span, 0.0), 1.0),)]
        mscale = 0.1 * math.log(factor) + 1.0
    return torch.tensor(f, dtype=torch.float64).to(torch.float32), mscale


def _rotary(stream, q, k, inv_freq, cu, lens, out, hq, hk, total, d, qs, ks, mscale, interleaved, transposed):
    device = (k if q is None else q).get_device()
    if out is None:
        qo = None if q is None else _empty((total, hq, d), dtype=_bf16, device=q.device)
        ko = None if k is None else _empty((total, hk, d), dtype=_bf16, device=k.device)
        qos, kos = hq * d, hk * d
    else:
        qo, ko = out
        if (q is None) != (qo is None) or (k is None) != (ko is None):
            raise ValueError("the outputs must hold q, or k, if and only if it is given")
        qos = 0 if qo is None else _tokens("the output of q", qo, device, q.shape)
        kos = 0 if ko is None else _tokens("the output of k", ko, device, k.shape)
    st = lib().fa_rotary(None if q is None else q.data_ptr(), None if k is None else k.data_ptr(),
                         None if qo is None else qo.data_ptr(), None if ko is None else ko.data_ptr(),
                         inv_freq.data_ptr(), cu.data_ptr(), None if lens is None else lens.data_ptr(), cu.shape[0] - 1,
                         hq, hk, total, d, 2 * inv_freq.shape[0], qs, ks, qos, kos, mscale, interleaved, transposed, stream)
    if st != 0:
        raise FAError(st, "fa_rotary")
    return qo, ko


def _turn(q, k, inv_freq, cu, lens, interleaved, mscale, out, stream, transposed):
    if q is None and k is None:
        raise ValueError("q or k must be given")
    some = k if q is None else q
    device = _first("k" if q is None else "q", some)
    total, hq, d = some.shape
    hk = qs = ks = 0
    if q is not None:
        qs = _tokens("q", q, device, q.shape)
    else:
        hq = 0
    if k is not None:
        if k.dim() != 3 or k.shape[0] != total or k.shape[1] < 1 or k.shape[2] != d:
            raise ValueError(f"k must have the shape [{total}, kv heads, {d}]")
        hk = k.shape[1]
        ks = _tokens("k", k, device, k.shape)
    n = cu.shape
    if not (len(n) == 1 and n[0] >= 2 and cu.dtype is _i32 and inv_freq.dim() == 1 and inv_freq.dtype is _f32
            and cu.is_contiguous() and inv_freq.is_contiguous() and cu.get_device() == inv_freq.get_device() == device):
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must hold a frequency for each pair")
        _packed("inv_freq", inv_freq, inv_freq.shape, device, _f32)
        _ints("cu", cu, n, device)
        raise ValueError("cu must hold the row offsets of one sequence at least")
    if lens is not None:
        _ints("lens", lens, (n[0] - 1,), device)
    s = _here(device, stream)
    if s is not None:
        return _rotary(s, q, k, inv_freq, cu, lens, out, hq, hk, total, d, qs, ks, float(mscale), 1 if interleaved else 0,
                       transposed)
    with _on(device, stream):
        return _rotary(_current_stream(), q, k, inv_freq, cu, lens, out, hq, hk, total, d, qs, ks, float(mscale),
                       1 if interleaved else 0, transposed)


def rotary(q, k, inv_freq, cu, lens=None, interleaved: bool = False, mscale: float = 1.0, out=None, stream=None):
    """q [total, Hq, d] and k [total, Hkv, d] (bf16, CUDA; tokens may be
    strided; either may be None) turned by their places: row i of sequence b is
    at lens[b] - n_b + i (lens int32 [B], the lengths with the new tokens, as
    cache_append takes them), or at i without lens; cu int32 [B + 1] row offsets;
    inv_freq fp32 [rot / 2] on the device, for the first rot values of a head
    (see fa.h fa_rotary and rotary_frequencies). out: a pair of tensors, (q, k)
    themselves for in place; new ones otherwise. Returns the outputs."""
    return _turn(q, k, inv_freq, cu, lens, interleaved, mscale, out, stream, 0)


def rotary_backward(dq, dk, inv_freq, cu, lens=None, interleaved: bool = False, mscale: float = 1.0, out=None,
                    stream=None):
    """The gradients of rotary's inputs from those of its outputs (bf16): the
    transposed turn, with the arguments that rotary had."""
    return _turn(dq, dk, inv_freq, cu, lens, interleaved, mscale, out, stream, 1)
