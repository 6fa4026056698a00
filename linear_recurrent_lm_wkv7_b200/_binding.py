"""ctypes binding of libwkv7.so (include/wkv7.h).

Argument marshalling only: tensors are passed as raw device pointers, dtype
codes are derived from the tensors, and the current torch CUDA stream is used
unless one is given.  Every call runs in the CUDA library; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libwkv7.so")

WKV7_F32 = 0
WKV7_BF16 = 1

STATUS = {
    0: "WKV7_OK",
    -1: "WKV7_ERR_INVALID_ARG",
    -2: "WKV7_ERR_UNSUPPORTED",
    -3: "WKV7_ERR_MISALIGNED",
    -4: "WKV7_ERR_CUDA",
    -5: "WKV7_ERR_DEVICE_TIMEOUT",
    -6: "WKV7_ERR_DEVICE_BOUNDS",
    -7: "WKV7_ERR_SCRATCH_LIMIT",
    -8: "WKV7_ERR_DECAY_RANGE",
}
# every symbol include/wkv7.h declares
EXPORTS = (
    "wkv7_forward",
    "wkv7_forward_gated",
    "wkv7_forward_fused",
    "wkv7_forward_long",
    "wkv7_forward_long_workspace_bytes",
    "wkv7_decode_step",
    "wkv7_decode_step_fused",
    "wkv7_backward",
    "wkv7_backward_workspace_bytes",
    "wkv7_backward_noalloc",
    "wkv7_state_map",
    "wkv7_state_apply",
    "wkv7_causal_conv",
    "wkv7_causal_conv_step",
    "wkv7_causal_conv_backward",
    "wkv7_causal_conv_backward_workspace_bytes",
    "wkv7_selective_scan",
    "wkv7_selective_scan_step",
    "wkv7_selective_scan_backward",
    "wkv7_selective_scan_backward_workspace_bytes",
    "wkv7_selective_scan_workspace_bytes",
    "wkv7_group_norm",
    "wkv7_group_norm_workspace_bytes",
    "wkv7_group_norm_backward",
    "wkv7_group_norm_backward_workspace_bytes",
    "wkv7_status_string",
    "wkv7_get_device_status",
    "wkv7_debug_expire_wait",
    "wkv7_version",
)


class Wkv7Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_lib().wkv7_status_string(status).decode()})")


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python linear_recurrent_lm_wkv7_b200/build.py`")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i = ctypes.c_void_p, ctypes.c_int
        lib.wkv7_forward.argtypes = [vp] * 9 + [i] * 4 + [vp, i, i, vp]
        lib.wkv7_forward.restype = i
        lib.wkv7_forward_gated.argtypes = [vp] * 11 + [i] * 4 + [vp, i, i, vp]
        lib.wkv7_forward_gated.restype = i
        lib.wkv7_forward_fused.argtypes = [vp] * 10 + [i] * 5 + [vp, i, i, vp]
        lib.wkv7_forward_fused.restype = i
        lib.wkv7_decode_step_fused.argtypes = [vp] * 10 + [i] * 4 + [i, i, vp]
        lib.wkv7_decode_step_fused.restype = i
        lib.wkv7_backward.argtypes = [vp] * 17 + [ctypes.c_size_t] + [i] * 4 + [vp, i, i, vp]
        lib.wkv7_backward.restype = i
        lib.wkv7_backward_workspace_bytes.argtypes = [i] * 5
        lib.wkv7_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.wkv7_backward_noalloc.argtypes = [vp] * 16 + [i] * 4 + [vp, i, i, vp]
        lib.wkv7_backward_noalloc.restype = i
        lib.wkv7_forward_long.argtypes = [vp] * 10 + [ctypes.c_size_t] + [i] * 4 + [i, i, vp]
        lib.wkv7_forward_long.restype = i
        lib.wkv7_forward_long_workspace_bytes.argtypes = [i] * 4
        lib.wkv7_forward_long_workspace_bytes.restype = ctypes.c_size_t
        lib.wkv7_state_map.argtypes = [vp] * 8 + [i] * 4 + [vp, i, i, vp]
        lib.wkv7_state_map.restype = i
        lib.wkv7_state_apply.argtypes = [vp] * 4 + [i, i, vp]
        lib.wkv7_state_apply.restype = i
        lib.wkv7_decode_step.argtypes = [vp] * 9 + [i] * 3 + [i, i, vp]
        lib.wkv7_decode_step.restype = i
        ll, sz, f = ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        lib.wkv7_causal_conv.argtypes = [vp, ll, vp, vp, vp, vp, ll, vp] + [i] * 4 + [vp, i, i, vp]
        lib.wkv7_causal_conv.restype = i
        lib.wkv7_causal_conv_step.argtypes = [vp, ll, vp, vp, vp, vp, ll, vp] + [i] * 5 + [vp]
        lib.wkv7_causal_conv_step.restype = i
        lib.wkv7_causal_conv_backward.argtypes = ([vp, ll, vp, vp, vp, vp, ll, vp, vp, ll, vp, vp, vp, vp, sz] +
                                                  [i] * 4 + [vp, i, i, vp])
        lib.wkv7_causal_conv_backward.restype = i
        lib.wkv7_causal_conv_backward_workspace_bytes.argtypes = [i] * 5
        lib.wkv7_causal_conv_backward_workspace_bytes.restype = sz
        lib.wkv7_selective_scan.argtypes = ([vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, vp, vp, ll, vp, vp, sz] +
                                            [i] * 6 + [vp, i, i, i, vp])
        lib.wkv7_selective_scan.restype = i
        lib.wkv7_selective_scan_step.argtypes = ([vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, vp, vp, ll, vp] +
                                                 [i] * 8 + [vp])
        lib.wkv7_selective_scan_step.restype = i
        lib.wkv7_selective_scan_workspace_bytes.argtypes = [i] * 6
        lib.wkv7_selective_scan_workspace_bytes.restype = sz
        lib.wkv7_selective_scan_backward.argtypes = ([vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, vp, vp, ll, vp, vp,
                                                      ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, vp, vp, sz] + [i] * 6 +
                                                     [vp, i, i, i, vp])
        lib.wkv7_selective_scan_backward.restype = i
        lib.wkv7_selective_scan_backward_workspace_bytes.argtypes = [i] * 8
        lib.wkv7_selective_scan_backward_workspace_bytes.restype = sz
        lib.wkv7_group_norm.argtypes = [vp, ll, vp, vp, vp, ll, vp, vp, sz] + [i] * 4 + [f, i, i, vp]
        lib.wkv7_group_norm.restype = i
        lib.wkv7_group_norm_backward.argtypes = [vp, ll, vp, vp, vp, vp, ll, vp, ll, vp, vp, vp, sz] + [i] * 6 + [vp]
        lib.wkv7_group_norm_backward.restype = i
        for name in ("wkv7_group_norm_workspace_bytes", "wkv7_group_norm_backward_workspace_bytes"):
            getattr(lib, name).argtypes = [i] * 5
            getattr(lib, name).restype = sz
        lib.wkv7_status_string.argtypes = [i]
        lib.wkv7_status_string.restype = ctypes.c_char_p
        lib.wkv7_get_device_status.argtypes = [vp]
        lib.wkv7_get_device_status.restype = i
        lib.wkv7_debug_expire_wait.argtypes = [i, vp]
        lib.wkv7_debug_expire_wait.restype = i
        lib.wkv7_version.argtypes = []
        lib.wkv7_version.restype = i
        _LIB = lib
    return _LIB


def _dtype_code(t):
    import torch

    if t.dtype == torch.float32:
        return WKV7_F32
    if t.dtype == torch.bfloat16:
        return WKV7_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def wkv7_forward(r, w_log, k, v, a, b, s0, y, sT, B, T, H, D, seq_offsets=None, stream=None):
    """Enqueue the chunked prefill (see include/wkv7.h).  Raises Wkv7Error on a
    non-OK status."""
    st = _lib().wkv7_forward(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(s0), _ptr(y),
                             _ptr(sT), int(B), int(T), int(H), int(D), _ptr(seq_offsets), _dtype_code(r),
                             _dtype_code(w_log), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_forward")


def wkv7_forward_gated(r, w_log, k, v, a, b, s0, r_k, g, z, sT, B, T, H, D, seq_offsets=None, stream=None):
    """Enqueue the prefill with the gated read-out (see include/wkv7.h)."""
    st = _lib().wkv7_forward_gated(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(s0), _ptr(r_k),
                                   _ptr(g), _ptr(z), _ptr(sT), int(B), int(T), int(H), int(D), _ptr(seq_offsets),
                                   _dtype_code(r), _dtype_code(w_log), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_forward_gated")


def wkv7_forward_fused(r, w_log, k, v, a_lr, s0, r_k, g, out, sT, B, T, H, H_kv, D, seq_offsets=None, stream=None):
    """Enqueue the prefill with the fused prologue (and the gated read-out when
    r_k and g are given); see include/wkv7.h."""
    st = _lib().wkv7_forward_fused(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a_lr), _ptr(s0), _ptr(r_k), _ptr(g),
                                   _ptr(out), _ptr(sT), int(B), int(T), int(H), int(H_kv), int(D), _ptr(seq_offsets),
                                   _dtype_code(r), _dtype_code(w_log), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_forward_fused")


def wkv7_decode_step_fused(r, w_log, k, v, a_lr, s_in, r_k, g, out, s_out, B, H, H_kv, D, stream=None):
    """Enqueue one decoding step with the fused prologue (and the gated read-out
    when r_k and g are given); see include/wkv7.h."""
    st = _lib().wkv7_decode_step_fused(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a_lr), _ptr(s_in), _ptr(r_k),
                                       _ptr(g), _ptr(out), _ptr(s_out), int(B), int(H), int(H_kv), int(D),
                                       _dtype_code(r), _dtype_code(w_log), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_decode_step_fused")


def wkv7_forward_long_workspace_bytes(B, T, H, D) -> int:
    return int(_lib().wkv7_forward_long_workspace_bytes(int(B), int(T), int(H), int(D)))


def wkv7_forward_long(r, w_log, k, v, a, b, s0, y, sT, workspace, B, T, H, D, stream=None):
    """Enqueue the two-phase prefill for long sequences (see include/wkv7.h)."""
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib().wkv7_forward_long(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(s0), _ptr(y),
                                  _ptr(sT), _ptr(workspace), int(nbytes), int(B), int(T), int(H), int(D),
                                  _dtype_code(r), _dtype_code(w_log), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_forward_long")


def wkv7_backward_workspace_bytes(B, T, H, D, packed) -> int:
    return int(_lib().wkv7_backward_workspace_bytes(int(B), int(T), int(H), int(D), 1 if packed else 0))


def wkv7_backward(r, w_log, k, v, a, b, s0, dy, dsT, dr, dw_log, dk, dv, da, db, ds0, workspace, B, T, H, D,
                  seq_offsets=None, stream=None):
    """Enqueue the backward of the recurrence (see include/wkv7.h)."""
    nbytes = workspace.numel() * workspace.element_size()
    st = _lib().wkv7_backward(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(s0), _ptr(dy),
                              _ptr(dsT), _ptr(dr), _ptr(dw_log), _ptr(dk), _ptr(dv), _ptr(da), _ptr(db), _ptr(ds0),
                              _ptr(workspace), int(nbytes), int(B), int(T), int(H), int(D), _ptr(seq_offsets),
                              _dtype_code(r), _dtype_code(w_log), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_backward")


def wkv7_backward_noalloc(r, w_log, k, v, a, b, s0, dy, dsT, dr, dw_log, dk, dv, da, db, ds0, B, T, H, D,
                          seq_offsets=None, stream=None):
    """Enqueue the backward with the library's fixed scratch: for callers that
    cannot allocate device memory at the call (see include/wkv7.h for the 16 MiB
    limit and the rule that overlapping calls must be ordered)."""
    st = _lib().wkv7_backward_noalloc(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(s0), _ptr(dy),
                                      _ptr(dsT), _ptr(dr), _ptr(dw_log), _ptr(dk), _ptr(dv), _ptr(da), _ptr(db),
                                      _ptr(ds0), int(B), int(T), int(H), int(D), _ptr(seq_offsets), _dtype_code(r),
                                      _dtype_code(w_log), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_backward_noalloc")


def wkv7_state_map(r, w_log, k, v, a, b, M, Q, B, T, H, D, seq_offsets=None, stream=None):
    """Enqueue the affine map of a token range (see include/wkv7.h): S_end = S_start M + Q.
    M or Q may be None (not computed)."""
    st = _lib().wkv7_state_map(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(M), _ptr(Q), int(B),
                               int(T), int(H), int(D), _ptr(seq_offsets), _dtype_code(r), _dtype_code(w_log),
                               _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_state_map")


def wkv7_state_apply(S_in, M, Q, S_out, n_units, D, stream=None):
    """Enqueue S_out = S_in M + Q over n_units states (S_in None: a zero state)."""
    st = _lib().wkv7_state_apply(_ptr(S_in), _ptr(M), _ptr(Q), _ptr(S_out), int(n_units), int(D), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_state_apply")


def wkv7_decode_step(r, w_log, k, v, a, b, s_in, y, s_out, B, H, D, stream=None):
    """Enqueue one decoding step (see include/wkv7.h)."""
    st = _lib().wkv7_decode_step(_ptr(r), _ptr(w_log), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(s_in), _ptr(y),
                                 _ptr(s_out), int(B), int(H), int(D), _dtype_code(r), _dtype_code(w_log),
                                 _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_decode_step")


# ---- causal convolution, selective scan, group norm: rows at a stride
#
# These calls check types, shapes, strides and devices of every tensor.  A single token
# per sequence takes the GPU a few microseconds, so the checks are written to be quick:
# one function call per tensor, and none of torch's slower queries.
WKV7_ACT = {None: 0, "none": 0, "silu": 1}


class _Runtime:
    """What the calls use of torch, looked up once.  The current stream is asked for by the name
    that torch's own code generators use: 0.07 us, where ``torch.cuda.current_stream(dev).cuda_stream``
    takes 1.3, of a call of 11."""

    def __init__(self):
        import torch

        self.f32, self.i32 = torch.float32, torch.int32
        self.codes = {torch.float32: WKV7_F32, torch.bfloat16: WKV7_BF16}
        self.device = torch.cuda.device
        self.current_device = torch._C._cuda_getDevice  # CUDA is set up: a tensor is on it
        self.raw_stream = torch._C._cuda_getCurrentRawStream


_RT = None


def _runtime():
    global _RT
    if _RT is None:
        _RT = _Runtime()
    return _RT


def _act(act):
    try:
        return WKV7_ACT[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {sorted(k for k in WKV7_ACT if k)}, not {act!r}") from None


def _code(t):
    c = _runtime().codes.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return c


def _row_ld(t, lead, width, name):
    """The row stride, in elements, of a tensor whose first ``lead`` dimensions number
    rows of ``width`` elements; the other dimensions have to be contiguous."""
    if t.is_contiguous():
        # of one row or none any stride that covers it will do
        return width if t.numel() > width else -(-width // 8) * 8
    shape, stride = t.shape, t.stride()
    inner = 1
    for k in range(len(shape) - 1, lead - 1, -1):
        if shape[k] != 1 and stride[k] != inner:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        inner *= shape[k]
    ld, rows = width, 1
    for k in range(lead - 1, -1, -1):
        if shape[k] == 1:
            continue
        if rows == 1:
            ld = stride[k]
        elif stride[k] != ld * rows:
            raise ValueError(f"{name}: the rows must lie at one stride")
        rows *= shape[k]
    return ld if rows > 1 else -(-width // 8) * 8


def _wrong(t, name, dtype, shape, dev):
    """Raises what is wrong with a tensor that did not pass a check."""
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _flat(t, name, dtype, shape, dev):
    """The pointer of a contiguous tensor of a given type and shape, or of none."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _wrong(t, name, dtype, shape, dev)
    return t.data_ptr()


_INT = 2 ** 31 - 1  # the library's sizes are ints, and ctypes would cut larger ones


def _rows(t, name, dtype, shape, lead, width, dev):
    """The pointer and the row stride of rows of ``width`` elements."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _wrong(t, name, dtype, shape, dev)
    if shape[0] > _INT or shape[lead - 1] > _INT or width > _INT:
        raise ValueError(f"{name}: every size must be below 2^31, not {tuple(shape)}")
    if lead == 1 and shape[0] > 1:  # the usual slice of a step or of packed rows
        st = t.stride()
        if st[-1] == 1 and (len(st) == 2 or st[1] == shape[2]):
            return t.data_ptr(), st[0]
    return t.data_ptr(), _row_ld(t, lead, width, name)


def _space(t, dev):
    """The pointer and the bytes of a workspace, or of none."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        _wrong(t, "workspace", t.dtype, t.shape, dev)
    return t.data_ptr(), t.numel() * t.element_size()


def _dev(t):
    """The ordinal of the device that a call runs on."""
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if _RT is None:
        _runtime()
    return dev


def _call(dev, stream, fn, args, where):
    """Calls the library with device ``dev`` current and raises on a status."""
    rt = _RT
    if stream is None:
        stream = rt.raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if rt.current_device() == dev:
        st = fn(*args, stream)
    else:
        with rt.device(dev):
            st = fn(*args, stream)
    if st:
        raise Wkv7Error(st, where)


def wkv7_causal_conv(x, w, bias, s0, y, sT, B, T, C, W, seq_offsets=None, act=None, stream=None):
    """Enqueue the causal convolution (see include/wkv7.h).  x and y may be slices of
    wider rows."""
    dev, io, code = _dev(x), x.dtype, _code(x)
    f32 = _RT.f32
    lead = (B, T) if seq_offsets is None else (T,)
    px, ldx = _rows(x, "x", io, lead + (C,), len(lead), C, dev)
    py, ldy = _rows(y, "y", io, lead + (C,), len(lead), C, dev)
    _call(dev, stream, _lib().wkv7_causal_conv,
          (px, ldx, _flat(w, "w", f32, (C, W), dev), _flat(bias, "bias", f32, (C,), dev),
           _flat(s0, "s0", io, (B, W - 1, C), dev), py, ldy, _flat(sT, "sT", io, (B, W - 1, C), dev), B, T, C, W,
           _flat(seq_offsets, "seq_offsets", _RT.i32, (B + 1,), dev), _act(act), code), "wkv7_causal_conv")


def wkv7_causal_conv_step(x, w, bias, s_in, y, s_out, B, C, W, act=None, stream=None):
    """Enqueue one token per sequence of the causal convolution (see include/wkv7.h)."""
    dev, io, code = _dev(x), x.dtype, _code(x)
    f32 = _RT.f32
    shape, st = (B, C), (B, W - 1, C)
    px, ldx = _rows(x, "x", io, shape, 1, C, dev)
    py, ldy = _rows(y, "y", io, shape, 1, C, dev)
    ps = _flat(s_in, "s_in", io, st, dev)
    pt = ps if s_out is s_in else _flat(s_out, "s_out", io, st, dev)
    _call(dev, stream, _lib().wkv7_causal_conv_step,
          (px, ldx, _flat(w, "w", f32, (C, W), dev), _flat(bias, "bias", f32, (C,), dev),
           ps, py, ldy, pt, B, C, W, _act(act), code), "wkv7_causal_conv_step")


def wkv7_causal_conv_backward_workspace_bytes(B, T, C, W, packed) -> int:
    return int(_lib().wkv7_causal_conv_backward_workspace_bytes(B, T, C, W, 1 if packed else 0))


def wkv7_causal_conv_backward(x, w, bias, s0, dy, dsT, dx, dw, dbias, ds0, workspace, B, T, C, W, seq_offsets=None,
                              act=None, stream=None):
    """Enqueue the gradient of the causal convolution (see include/wkv7.h)."""
    dev, io, code = _dev(x), x.dtype, _code(x)
    f32 = _RT.f32
    lead = (B, T) if seq_offsets is None else (T,)
    k, shape, st = len(lead), lead + (C,), (B, W - 1, C)
    px, ldx = _rows(x, "x", io, shape, k, C, dev)
    pdy, lddy = _rows(dy, "dy", io, shape, k, C, dev)
    pdx, lddx = _rows(dx, "dx", io, shape, k, C, dev)
    ws, nbytes = _space(workspace, dev)
    _call(dev, stream, _lib().wkv7_causal_conv_backward,
          (px, ldx, _flat(w, "w", f32, (C, W), dev), _flat(bias, "bias", f32, (C,), dev),
           _flat(s0, "s0", io, st, dev), pdy, lddy, _flat(dsT, "dsT", io, st, dev), pdx, lddx,
           _flat(dw, "dw", f32, (C, W), dev), _flat(dbias, "dbias", f32, (C,), dev), _flat(ds0, "ds0", io, st, dev),
           ws, nbytes, B, T, C, W, _flat(seq_offsets, "seq_offsets", _RT.i32, (B + 1,), dev), _act(act), code),
          "wkv7_causal_conv_backward")


def _scan_inputs(x, dt, A, Bm, Cm, D_skip, dt_bias, lead, H, D, N, G, dev):
    """The leading arguments that the scan's calls share: x to dt_bias."""
    f32, io, k, hs, bs = _RT.f32, x.dtype, len(lead), (H,), lead + (G, N)
    px, ldx = _rows(x, "x", io, lead + (H, D), k, H * D, dev)
    pt, ldt = _rows(dt, "dt", dt.dtype, lead + hs, k, H, dev)
    pb, ldb = _rows(Bm, "Bm", io, bs, k, G * N, dev)
    pc, ldc = _rows(Cm, "Cm", io, bs, k, G * N, dev)
    return (px, ldx, pt, ldt, _flat(A, "A", f32, hs, dev), pb, ldb, pc, ldc, _flat(D_skip, "D_skip", f32, hs, dev),
            _flat(dt_bias, "dt_bias", f32, hs, dev))


def wkv7_selective_scan_workspace_bytes(B, T, H, D, N, packed) -> int:
    return int(_lib().wkv7_selective_scan_workspace_bytes(B, T, H, D, N, 1 if packed else 0))


def wkv7_selective_scan(x, dt, A, Bm, Cm, D_skip, dt_bias, s0, y, sT, workspace, B, T, H, D, N, G, seq_offsets=None,
                        dt_softplus=True, stream=None):
    """Enqueue the selective scan (see include/wkv7.h).  x, dt, Bm, Cm and y may be
    slices of wider rows."""
    dev, code, dtc = _dev(x), _code(x), _code(dt)
    f32 = _RT.f32
    lead = (B, T) if seq_offsets is None else (T,)
    ins = _scan_inputs(x, dt, A, Bm, Cm, D_skip, dt_bias, lead, H, D, N, G, dev)
    ws, nbytes = _space(workspace, dev)
    _call(dev, stream, _lib().wkv7_selective_scan,
          ins + (_flat(s0, "s0", f32, (B, H, D, N), dev),) +
          _rows(y, "y", x.dtype, lead + (H, D), len(lead), H * D, dev) +
          (_flat(sT, "sT", f32, (B, H, D, N), dev), ws, nbytes, B, T, H, D, N, G,
           _flat(seq_offsets, "seq_offsets", _RT.i32, (B + 1,), dev), 1 if dt_softplus else 0, code, dtc),
          "wkv7_selective_scan")


def wkv7_selective_scan_step(x, dt, A, Bm, Cm, D_skip, dt_bias, s_in, y, s_out, B, H, D, N, G, dt_softplus=True,
                             stream=None):
    """Enqueue one token per sequence of the selective scan (see include/wkv7.h)."""
    dev, code, dtc = _dev(x), _code(x), _code(dt)
    st = (B, H, D, N)
    ps = _flat(s_in, "s_in", _RT.f32, st, dev)
    pt = ps if s_out is s_in else _flat(s_out, "s_out", _RT.f32, st, dev)
    _call(dev, stream, _lib().wkv7_selective_scan_step,
          (*_scan_inputs(x, dt, A, Bm, Cm, D_skip, dt_bias, (B,), H, D, N, G, dev), ps,
           *_rows(y, "y", x.dtype, (B, H, D), 1, H * D, dev), pt, B, H, D, N, G, 1 if dt_softplus else 0, code, dtc),
          "wkv7_selective_scan_step")


def wkv7_selective_scan_backward_workspace_bytes(B, T, H, D, N, G, io_dtype, packed) -> int:
    return int(_lib().wkv7_selective_scan_backward_workspace_bytes(B, T, H, D, N, G, io_dtype, 1 if packed else 0))


def wkv7_selective_scan_backward(x, dt, A, Bm, Cm, D_skip, dt_bias, s0, dy, dsT, dx, ddt, dA, dB, dC, dD, ddt_bias,
                                 ds0, workspace, B, T, H, D, N, G, seq_offsets=None, dt_softplus=True, stream=None):
    """Enqueue the gradient of the selective scan (see include/wkv7.h).  dx, dB and dC may
    be column slices of one buffer, for the convolution's backward to take."""
    dev, code, dtc = _dev(x), _code(x), _code(dt)
    f32 = _RT.f32
    lead = (B, T) if seq_offsets is None else (T,)
    k, io, st = len(lead), x.dtype, (B, H, D, N)
    ins = _scan_inputs(x, dt, A, Bm, Cm, D_skip, dt_bias, lead, H, D, N, G, dev)
    ws, nbytes = _space(workspace, dev)
    _call(dev, stream, _lib().wkv7_selective_scan_backward,
          ins + (_flat(s0, "s0", f32, st, dev),) + _rows(dy, "dy", io, lead + (H, D), k, H * D, dev) +
          (_flat(dsT, "dsT", f32, st, dev),) + _rows(dx, "dx", io, lead + (H, D), k, H * D, dev) +
          _rows(ddt, "ddt", dt.dtype, lead + (H,), k, H, dev) + (_flat(dA, "dA", f32, (H,), dev),) +
          _rows(dB, "dB", io, lead + (G, N), k, G * N, dev) + _rows(dC, "dC", io, lead + (G, N), k, G * N, dev) +
          (_flat(dD, "dD", f32, (H,), dev), _flat(ddt_bias, "ddt_bias", f32, (H,), dev),
           _flat(ds0, "ds0", f32, st, dev), ws, nbytes, B, T, H, D, N, G,
           _flat(seq_offsets, "seq_offsets", _RT.i32, (B + 1,), dev), 1 if dt_softplus else 0, code, dtc),
          "wkv7_selective_scan_backward")


def _norm_lead(x, N, L):
    return (N,) if x.dim() == 2 and L == 1 else (N, L)


def wkv7_group_norm_workspace_bytes(N, L, C, G, io_dtype) -> int:
    return int(_lib().wkv7_group_norm_workspace_bytes(N, L, C, G, io_dtype))


def wkv7_group_norm(x, weight, bias, y, stats, workspace, N, L, C, G, eps=1e-5, act=None, stream=None):
    """Enqueue the group norm (see include/wkv7.h)."""
    dev, io, code = _dev(x), x.dtype, _code(x)
    f32 = _RT.f32
    lead = _norm_lead(x, N, L)
    px, ldx = _rows(x, "x", io, lead + (C,), len(lead), C, dev)
    py, ldy = _rows(y, "y", io, lead + (C,), len(lead), C, dev)
    ws, nbytes = _space(workspace, dev)
    _call(dev, stream, _lib().wkv7_group_norm,
          (px, ldx, _flat(weight, "weight", f32, (C,), dev), _flat(bias, "bias", f32, (C,), dev), py, ldy,
           _flat(stats, "stats", f32, (N, G, 2), dev), ws, nbytes, N, L, C, G, eps, _act(act), code),
          "wkv7_group_norm")


def wkv7_group_norm_backward_workspace_bytes(N, L, C, G, io_dtype) -> int:
    return int(_lib().wkv7_group_norm_backward_workspace_bytes(N, L, C, G, io_dtype))


def wkv7_group_norm_backward(x, weight, bias, stats, dy, dx, dweight, dbias, workspace, N, L, C, G, act=None,
                             stream=None):
    """Enqueue the gradient of the group norm (see include/wkv7.h)."""
    dev, io, code = _dev(x), x.dtype, _code(x)
    f32 = _RT.f32
    lead = _norm_lead(x, N, L)
    k, shape = len(lead), lead + (C,)
    px, ldx = _rows(x, "x", io, shape, k, C, dev)
    pdy, lddy = _rows(dy, "dy", io, shape, k, C, dev)
    pdx, lddx = _rows(dx, "dx", io, shape, k, C, dev)
    ws, nbytes = _space(workspace, dev)
    _call(dev, stream, _lib().wkv7_group_norm_backward,
          (px, ldx, _flat(weight, "weight", f32, (C,), dev), _flat(bias, "bias", f32, (C,), dev),
           _flat(stats, "stats", f32, (N, G, 2), dev), pdy, lddy, pdx, lddx, _flat(dweight, "dweight", f32, (C,), dev),
           _flat(dbias, "dbias", f32, (C,), dev), ws, nbytes, N, L, C, G, _act(act), code), "wkv7_group_norm_backward")


def wkv7_get_device_status(stream=None) -> int:
    return int(_lib().wkv7_get_device_status(_stream(stream)))


def wkv7_debug_expire_wait(spins: int, stream=None) -> None:
    st = _lib().wkv7_debug_expire_wait(int(spins), _stream(stream))
    if st != 0:
        raise Wkv7Error(st, "wkv7_debug_expire_wait")


def wkv7_status_string(status: int) -> str:
    return _lib().wkv7_status_string(int(status)).decode()


def wkv7_version() -> int:
    return int(_lib().wkv7_version())


def raw_call_forward(*args):
    """Direct C call with raw integer pointers (used by host-validation tests)."""
    return int(_lib().wkv7_forward(*args))


def raw_call_forward_long(*args):
    return int(_lib().wkv7_forward_long(*args))


def raw_call_forward_gated(*args):
    return int(_lib().wkv7_forward_gated(*args))


def raw_call_forward_fused(*args):
    return int(_lib().wkv7_forward_fused(*args))


def raw_call_decode_fused(*args):
    return int(_lib().wkv7_decode_step_fused(*args))


def raw_call_backward(*args):
    return int(_lib().wkv7_backward(*args))


def raw_call_backward_noalloc(*args):
    return int(_lib().wkv7_backward_noalloc(*args))


def raw_call_state_map(*args):
    return int(_lib().wkv7_state_map(*args))


def raw_call_state_apply(*args):
    return int(_lib().wkv7_state_apply(*args))


def raw_call_decode(*args):
    return int(_lib().wkv7_decode_step(*args))
