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
WKV7_ACT = {None: 0, "none": 0, "silu": 1}


def _act(act):
    try:
        return WKV7_ACT[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {sorted(k for k in WKV7_ACT if k)}, not {act!r}") from None


def _code(t):
    import torch

    dt = t.dtype
    if dt is torch.bfloat16:
        return WKV7_BF16
    if dt is torch.float32:
        return WKV7_F32
    raise TypeError(f"unsupported dtype {dt}")


def _row_ld(t, lead, width, name):
    """The row stride, in elements, of a tensor whose first ``lead`` dimensions number
    rows of ``width`` elements; the other dimensions have to be contiguous."""
    shape, stride = t.shape, t.stride()
    if 0 in shape:  # no rows: any stride that covers one will do
        return -(-width // 8) * 8
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


def _at(device, **tensors):
    """The raw pointers of tensors that may be None, all on one device."""
    out = []
    for name, t in tensors.items():
        if t is None:
            out.append(None)
            continue
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")
        out.append(t.data_ptr())
    return out


def _need(t, name, dtype, shape):
    """An optional contiguous tensor of a given type and shape."""
    if t is None:
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _cuda(t):
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    return t.device


def _call(device, stream, fn, args, where):
    """Calls the library with ``device`` current and raises on a status."""
    import torch

    if stream is None:
        stream = torch.cuda.current_stream(device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == device.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != 0:
        raise Wkv7Error(st, where)


def _packed(seq_offsets, B):
    import torch

    _need(seq_offsets, "seq_offsets", torch.int32, (B + 1,))


def _like(t, ref, name):
    if t.dtype is not ref.dtype:
        raise TypeError(f"{name} must be {ref.dtype}, not {t.dtype}")
    if t.shape != ref.shape:
        raise ValueError(f"{name} must have the shape {tuple(ref.shape)}, not {tuple(t.shape)}")


def _leading(t, inner, B, T, seq_offsets, name):
    """How many dimensions number rows ([B, T, ..] or packed [T, ..]), after a check."""
    lead = (T,) if seq_offsets is not None else (B, T)
    if tuple(t.shape) != lead + tuple(inner):
        raise ValueError(f"{name} must have the shape {lead + tuple(inner)}, not {tuple(t.shape)}")
    return len(lead)


def wkv7_causal_conv(x, w, bias, s0, y, sT, B, T, C, W, seq_offsets=None, act=None, stream=None):
    """Enqueue the causal convolution (see include/wkv7.h).  x and y may be slices of
    wider rows."""
    import torch

    dev = _cuda(x)
    lead = _leading(x, (C,), B, T, seq_offsets, "x")
    _like(y, x, "y")
    _need(w, "w", torch.float32, (C, W))
    _need(bias, "bias", torch.float32, (C,))
    _need(s0, "s0", x.dtype, (B, W - 1, C))
    _need(sT, "sT", x.dtype, (B, W - 1, C))
    _packed(seq_offsets, B)
    px, pw, pb, p0, py, pT, po = _at(dev, x=x, w=w, bias=bias, s0=s0, y=y, sT=sT, seq_offsets=seq_offsets)
    _call(dev, stream, _lib().wkv7_causal_conv,
          (px, _row_ld(x, lead, C, "x"), pw, pb, p0, py, _row_ld(y, lead, C, "y"), pT, B, T, C, W, po, _act(act),
           _code(x)), "wkv7_causal_conv")


def wkv7_causal_conv_step(x, w, bias, s_in, y, s_out, B, C, W, act=None, stream=None):
    """Enqueue one token per sequence of the causal convolution (see include/wkv7.h)."""
    import torch

    dev = _cuda(x)
    if tuple(x.shape) != (B, C):
        raise ValueError(f"x must have the shape {(B, C)}, not {tuple(x.shape)}")
    _like(y, x, "y")
    _need(w, "w", torch.float32, (C, W))
    _need(bias, "bias", torch.float32, (C,))
    _need(s_in, "s_in", x.dtype, (B, W - 1, C))
    _need(s_out, "s_out", x.dtype, (B, W - 1, C))
    px, pw, pb, p0, py, pT = _at(dev, x=x, w=w, bias=bias, s_in=s_in, y=y, s_out=s_out)
    _call(dev, stream, _lib().wkv7_causal_conv_step,
          (px, _row_ld(x, 1, C, "x"), pw, pb, p0, py, _row_ld(y, 1, C, "y"), pT, B, C, W, _act(act), _code(x)),
          "wkv7_causal_conv_step")


def wkv7_causal_conv_backward_workspace_bytes(B, T, C, W, packed) -> int:
    return int(_lib().wkv7_causal_conv_backward_workspace_bytes(B, T, C, W, 1 if packed else 0))


def wkv7_causal_conv_backward(x, w, bias, s0, dy, dsT, dx, dw, dbias, ds0, workspace, B, T, C, W, seq_offsets=None,
                              act=None, stream=None):
    """Enqueue the gradient of the causal convolution (see include/wkv7.h)."""
    import torch

    dev = _cuda(x)
    lead = _leading(x, (C,), B, T, seq_offsets, "x")
    _like(dy, x, "dy")
    _like(dx, x, "dx")
    for t, name in ((w, "w"), (dw, "dw")):
        _need(t, name, torch.float32, (C, W))
    for t, name in ((bias, "bias"), (dbias, "dbias")):
        _need(t, name, torch.float32, (C,))
    for t, name in ((s0, "s0"), (dsT, "dsT"), (ds0, "ds0")):
        _need(t, name, x.dtype, (B, W - 1, C))
    _packed(seq_offsets, B)
    px, pw, pb, p0, pdy, pdT, pdx, pdw, pdb, pd0, ws, po = _at(
        dev, x=x, w=w, bias=bias, s0=s0, dy=dy, dsT=dsT, dx=dx, dw=dw, dbias=dbias, ds0=ds0, workspace=workspace,
        seq_offsets=seq_offsets)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call(dev, stream, _lib().wkv7_causal_conv_backward,
          (px, _row_ld(x, lead, C, "x"), pw, pb, p0, pdy, _row_ld(dy, lead, C, "dy"), pdT, pdx,
           _row_ld(dx, lead, C, "dx"), pdw, pdb, pd0, ws, nbytes, B, T, C, W, po, _act(act), _code(x)),
          "wkv7_causal_conv_backward")


def _scan_inputs(x, dt, A, Bm, Cm, D_skip, dt_bias, B, T, H, D, N, G, seq_offsets, step):
    import torch

    if step:
        seq_offsets, lead = None, 1
        for t, inner, name in ((x, (H, D), "x"), (dt, (H,), "dt"), (Bm, (G, N), "Bm"), (Cm, (G, N), "Cm")):
            if tuple(t.shape) != (B,) + inner:
                raise ValueError(f"{name} must have the shape {(B,) + inner}, not {tuple(t.shape)}")
    else:
        lead = _leading(x, (H, D), B, T, seq_offsets, "x")
        _leading(dt, (H,), B, T, seq_offsets, "dt")
        _leading(Bm, (G, N), B, T, seq_offsets, "Bm")
        _leading(Cm, (G, N), B, T, seq_offsets, "Cm")
    if Bm.dtype is not x.dtype or Cm.dtype is not x.dtype:
        raise TypeError(f"Bm and Cm must be {x.dtype}, as x is")
    for t, name in ((A, "A"), (D_skip, "D_skip"), (dt_bias, "dt_bias")):
        _need(t, name, torch.float32, (H,))
    return (lead, _row_ld(x, lead, H * D, "x"), _row_ld(dt, lead, H, "dt"), _row_ld(Bm, lead, G * N, "Bm"),
            _row_ld(Cm, lead, G * N, "Cm"))


def wkv7_selective_scan_workspace_bytes(B, T, H, D, N, packed) -> int:
    return int(_lib().wkv7_selective_scan_workspace_bytes(B, T, H, D, N, 1 if packed else 0))


def wkv7_selective_scan(x, dt, A, Bm, Cm, D_skip, dt_bias, s0, y, sT, workspace, B, T, H, D, N, G, seq_offsets=None,
                        dt_softplus=True, stream=None):
    """Enqueue the selective scan (see include/wkv7.h).  x, dt, Bm, Cm and y may be
    slices of wider rows."""
    import torch

    dev = _cuda(x)
    lead, ldx, lddt, ldb, ldc = _scan_inputs(x, dt, A, Bm, Cm, D_skip, dt_bias, B, T, H, D, N, G, seq_offsets, False)
    _like(y, x, "y")
    _need(s0, "s0", torch.float32, (B, H, D, N))
    _need(sT, "sT", torch.float32, (B, H, D, N))
    _packed(seq_offsets, B)
    px, pdt, pA, pB, pC, pD, pb, p0, py, pT, ws, po = _at(
        dev, x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, D_skip=D_skip, dt_bias=dt_bias, s0=s0, y=y, sT=sT, workspace=workspace,
        seq_offsets=seq_offsets)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call(dev, stream, _lib().wkv7_selective_scan,
          (px, ldx, pdt, lddt, pA, pB, ldb, pC, ldc, pD, pb, p0, py, _row_ld(y, lead, H * D, "y"), pT, ws, nbytes, B,
           T, H, D, N, G, po, 1 if dt_softplus else 0, _code(x), _code(dt)), "wkv7_selective_scan")


def wkv7_selective_scan_step(x, dt, A, Bm, Cm, D_skip, dt_bias, s_in, y, s_out, B, H, D, N, G, dt_softplus=True,
                             stream=None):
    """Enqueue one token per sequence of the selective scan (see include/wkv7.h)."""
    import torch

    dev = _cuda(x)
    _, ldx, lddt, ldb, ldc = _scan_inputs(x, dt, A, Bm, Cm, D_skip, dt_bias, B, 1, H, D, N, G, None, True)
    _like(y, x, "y")
    _need(s_in, "s_in", torch.float32, (B, H, D, N))
    _need(s_out, "s_out", torch.float32, (B, H, D, N))
    px, pdt, pA, pB, pC, pD, pb, p0, py, pT = _at(dev, x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, D_skip=D_skip, dt_bias=dt_bias,
                                                  s_in=s_in, y=y, s_out=s_out)
    _call(dev, stream, _lib().wkv7_selective_scan_step,
          (px, ldx, pdt, lddt, pA, pB, ldb, pC, ldc, pD, pb, p0, py, _row_ld(y, 1, H * D, "y"), pT, B, H, D, N, G,
           1 if dt_softplus else 0, _code(x), _code(dt)), "wkv7_selective_scan_step")


def wkv7_selective_scan_backward_workspace_bytes(B, T, H, D, N, G, io_dtype, packed) -> int:
    return int(_lib().wkv7_selective_scan_backward_workspace_bytes(B, T, H, D, N, G, io_dtype, 1 if packed else 0))


def wkv7_selective_scan_backward(x, dt, A, Bm, Cm, D_skip, dt_bias, s0, dy, dsT, dx, ddt, dA, dB, dC, dD, ddt_bias,
                                 ds0, workspace, B, T, H, D, N, G, seq_offsets=None, dt_softplus=True, stream=None):
    """Enqueue the gradient of the selective scan (see include/wkv7.h).  dx, dB and dC may
    be column slices of one buffer, for the convolution's backward to take."""
    import torch

    dev = _cuda(x)
    lead, ldx, lddt, ldb, ldc = _scan_inputs(x, dt, A, Bm, Cm, D_skip, dt_bias, B, T, H, D, N, G, seq_offsets, False)
    for t, ref, name in ((dy, x, "dy"), (dx, x, "dx"), (ddt, dt, "ddt"), (dB, Bm, "dB"), (dC, Cm, "dC")):
        _like(t, ref, name)
    for t, name in ((dA, "dA"), (dD, "dD"), (ddt_bias, "ddt_bias")):
        _need(t, name, torch.float32, (H,))
    for t, name in ((s0, "s0"), (dsT, "dsT"), (ds0, "ds0")):
        _need(t, name, torch.float32, (B, H, D, N))
    _packed(seq_offsets, B)
    px, pdt, pA, pB, pC, pD, pb, p0, pdy, pdT = _at(dev, x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, D_skip=D_skip,
                                                    dt_bias=dt_bias, s0=s0, dy=dy, dsT=dsT)
    qx, qdt, qA, qB, qC, qD, qb, q0, ws, po = _at(dev, dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD, ddt_bias=ddt_bias,
                                                  ds0=ds0, workspace=workspace, seq_offsets=seq_offsets)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call(dev, stream, _lib().wkv7_selective_scan_backward,
          (px, ldx, pdt, lddt, pA, pB, ldb, pC, ldc, pD, pb, p0, pdy, _row_ld(dy, lead, H * D, "dy"), pdT, qx,
           _row_ld(dx, lead, H * D, "dx"), qdt, _row_ld(ddt, lead, H, "ddt"), qA, qB,
           _row_ld(dB, lead, G * N, "dB"), qC, _row_ld(dC, lead, G * N, "dC"), qD, qb, q0, ws, nbytes, B, T, H, D, N,
           G, po, 1 if dt_softplus else 0, _code(x), _code(dt)), "wkv7_selective_scan_backward")


def _norm_dims(x, N, L, C, name="x"):
    want = (N, C) if x.dim() == 2 and L == 1 else (N, L, C)
    if tuple(x.shape) != want:
        raise ValueError(f"{name} must have the shape {want}, not {tuple(x.shape)}")
    return len(want) - 1


def wkv7_group_norm_workspace_bytes(N, L, C, G, io_dtype) -> int:
    return int(_lib().wkv7_group_norm_workspace_bytes(N, L, C, G, io_dtype))


def wkv7_group_norm(x, weight, bias, y, stats, workspace, N, L, C, G, eps=1e-5, act=None, stream=None):
    """Enqueue the group norm (see include/wkv7.h)."""
    import torch

    dev = _cuda(x)
    lead = _norm_dims(x, N, L, C)
    _like(y, x, "y")
    _need(weight, "weight", torch.float32, (C,))
    _need(bias, "bias", torch.float32, (C,))
    _need(stats, "stats", torch.float32, (N, G, 2))
    px, pw, pb, py, ps, ws = _at(dev, x=x, weight=weight, bias=bias, y=y, stats=stats, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call(dev, stream, _lib().wkv7_group_norm,
          (px, _row_ld(x, lead, C, "x"), pw, pb, py, _row_ld(y, lead, C, "y"), ps, ws, nbytes, N, L, C, G, eps,
           _act(act), _code(x)), "wkv7_group_norm")


def wkv7_group_norm_backward_workspace_bytes(N, L, C, G, io_dtype) -> int:
    return int(_lib().wkv7_group_norm_backward_workspace_bytes(N, L, C, G, io_dtype))


def wkv7_group_norm_backward(x, weight, bias, stats, dy, dx, dweight, dbias, workspace, N, L, C, G, act=None,
                             stream=None):
    """Enqueue the gradient of the group norm (see include/wkv7.h)."""
    import torch

    dev = _cuda(x)
    lead = _norm_dims(x, N, L, C)
    _like(dy, x, "dy")
    _like(dx, x, "dx")
    for t, name in ((weight, "weight"), (bias, "bias"), (dweight, "dweight"), (dbias, "dbias")):
        _need(t, name, torch.float32, (C,))
    _need(stats, "stats", torch.float32, (N, G, 2))
    px, pw, pb, ps, pdy, pdx, pdw, pdb, ws = _at(dev, x=x, weight=weight, bias=bias, stats=stats, dy=dy, dx=dx,
                                                 dweight=dweight, dbias=dbias, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call(dev, stream, _lib().wkv7_group_norm_backward,
          (px, _row_ld(x, lead, C, "x"), pw, pb, ps, pdy, _row_ld(dy, lead, C, "dy"), pdx,
           _row_ld(dx, lead, C, "dx"), pdw, pdb, ws, nbytes, N, L, C, G, _act(act), _code(x)),
          "wkv7_group_norm_backward")


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
