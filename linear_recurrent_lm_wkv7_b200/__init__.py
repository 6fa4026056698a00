"""B200 (sm_100a) WKV-7 operator: chunked tensor-core prefill and streaming
decode step behind a C ABI (``include/wkv7.h``, ``libwkv7.so``).

The Python layer only marshals arguments to the CUDA library; importing the
package loads ``libwkv7.so`` and fails loudly if it has not been built.
Convenience wrappers ``forward``, ``forward_long``, ``forward_gated``, ``forward_fused``,
``decode_step``, ``decode_step_fused`` and ``backward`` allocate outputs with
torch and call the C entry points; ``forward_host`` runs the prefill on inputs
and outputs that live in pinned host memory, overlapping the copies with the
kernels.
"""
from __future__ import annotations

import functools

from ._binding import (  # noqa: F401
    EXPORTS,
    LIB_PATH,
    STATUS,
    WKV7_BF16,
    WKV7_F32,
    Wkv7Error,
    _code,
    _lib,
    wkv7_backward,
    wkv7_backward_noalloc,
    wkv7_backward_workspace_bytes,
    wkv7_causal_conv,
    wkv7_causal_conv_backward,
    wkv7_causal_conv_backward_workspace_bytes,
    wkv7_causal_conv_step,
    wkv7_debug_expire_wait,
    wkv7_decode_step,
    wkv7_decode_step_fused,
    wkv7_forward,
    wkv7_forward_fused,
    wkv7_forward_gated,
    wkv7_forward_long,
    wkv7_forward_long_workspace_bytes,
    wkv7_get_device_status,
    wkv7_group_norm,
    wkv7_group_norm_backward,
    wkv7_group_norm_backward_workspace_bytes,
    wkv7_group_norm_workspace_bytes,
    wkv7_selective_scan,
    wkv7_selective_scan_backward,
    wkv7_selective_scan_backward_workspace_bytes,
    wkv7_selective_scan_step,
    wkv7_selective_scan_workspace_bytes,
    wkv7_state_apply,
    wkv7_state_map,
    wkv7_status_string,
    wkv7_version,
)

_lib()  # load now: a missing or broken library is an import error, never a silent fallback


def forward(r, w_log, k, v, a, b, s0=None, seq_offsets=None, want_state=True, stream=None):
    """Chunked prefill.  Dense inputs are [B, T, H, D]; packed inputs are
    [T, H, D] with int32 ``seq_offsets`` [B+1] on the device.  Returns
    ``(y, sT)`` (``sT`` is None when ``want_state`` is false)."""
    import torch

    if seq_offsets is not None:
        T, H, D = r.shape
        B = seq_offsets.numel() - 1
    else:
        B, T, H, D = r.shape
    y = torch.empty_like(r)
    sT = torch.empty((B, H, D, D), dtype=torch.float32, device=r.device) if want_state else None
    wkv7_forward(r, w_log, k, v, a, b, s0, y, sT, B, T, H, D, seq_offsets, stream)
    return y, sT


def forward_long(r, w_log, k, v, a, b, s0=None, want_state=True, workspace=None, stream=None):
    """Two-phase prefill of a dense batch [B, T, H, D] (bf16 inputs) for few,
    long sequences: every chunk's state-independent work in parallel, then one
    state pass per (sequence, head).  ``workspace`` (a device tensor of at least
    ``wkv7_forward_long_workspace_bytes`` bytes) is allocated when not given.
    Returns ``(y, sT)`` like ``forward``."""
    import torch

    B, T, H, D = r.shape
    if workspace is None:
        nbytes = wkv7_forward_long_workspace_bytes(B, T, H, D)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=r.device)
    y = torch.empty_like(r)
    sT = torch.empty((B, H, D, D), dtype=torch.float32, device=r.device) if want_state else None
    wkv7_forward_long(r, w_log, k, v, a, b, s0, y, sT, workspace, B, T, H, D, stream)
    return y, sT


_HOST_STREAMS = {}
_INPUTS = ("r", "w_log", "k", "v", "a", "b")


def host_pieces(B, T, parts=4, t_parts=1):
    """How ``forward_host`` cuts a dense [B, T, ...] batch: returns ``(groups, bounds)``,
    sequence groups [b0, b1) and token bounds, so that each piece (group, [t0, t1))
    is contiguous in memory.  With ``t_parts`` > 1 every sequence is its own group
    and the token bounds are multiples of 64 (the chunk length), so a range
    continues exactly where the previous one stopped; otherwise there are ``parts``
    groups of whole sequences.  T = 0 gives one empty range."""
    t_parts = max(1, int(t_parts))
    nck = (T + 63) // 64
    bounds = sorted({min(T, 64 * (nck * j // t_parts)) for j in range(t_parts)} | {T})
    if T == 0:
        bounds = [0, 0]  # one empty piece: sT receives s0 (or zeros)
    if len(bounds) > 2:
        groups = [(b, b + 1) for b in range(B)]
    else:
        n = max(1, min(int(parts), B))
        groups = [(B * p // n, B * (p + 1) // n) for p in range(n)]
    return groups, bounds


def forward_host(host, dev, y_host, sT_host, s0=None, parts=4, t_parts=1, stream=None):
    """Prefill of a dense batch whose inputs and outputs live in pinned host memory.

    ``host``: pinned CPU tensors r, w_log, k, v, a, b of shape [B, T, H, D];
    ``dev``: device staging tensors of the same names and shapes plus ``y`` and
    ``sT`` ([B, H, D, D] fp32), allocated once by the caller; ``y_host``,
    ``sT_host``: pinned CPU outputs; ``s0``: optional device initial states.
    The batch is cut into pieces, each contiguous in memory: ``parts`` groups of
    whole sequences, or, with ``t_parts`` > 1 (for batches of few long
    sequences), every sequence cut into that many token ranges whose bounds are
    multiples of 64, a range continuing from the state the previous one left in
    ``dev["sT"]`` (updated in place).  Every piece costs a few host-side calls, so
    a handful of large pieces is best.
    The upload of one piece, the prefill of the previous and the download of the
    one before run on three CUDA streams at once, and the results equal one call
    over the whole batch.  Everything is ordered after ``stream`` (default: the
    current stream), which then waits for all of it: the call is asynchronous
    like a kernel launch on ``stream``.
    The three side streams are created once per device and shared by every call
    on that device.  Calls from several host threads at once are correct but
    their copies and kernels serialise on those streams; such calls must not
    share ``dev`` buffers (nothing orders one call's use of them against
    another's)."""
    import torch

    device = dev["r"].device
    st = stream if stream is not None else torch.cuda.current_stream(device)
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if idx not in _HOST_STREAMS:
        _HOST_STREAMS[idx] = tuple(torch.cuda.Stream(device) for _ in range(3))
    s_up, s_run, s_down = _HOST_STREAMS[idx]
    B, T, H, D = host["r"].shape
    groups, tb = host_pieces(B, T, parts, t_parts)
    start = torch.cuda.Event()
    start.record(st)
    for s_ in (s_up, s_run, s_down):
        s_.wait_event(start)
    for b0, b1 in groups:
        if b1 == b0:
            continue
        for j in range(len(tb) - 1):
            t0, t1 = tb[j], tb[j + 1]
            with torch.cuda.stream(s_up):
                for n in _INPUTS:
                    dev[n][b0:b1, t0:t1].copy_(host[n][b0:b1, t0:t1], non_blocking=True)
            up = torch.cuda.Event()
            up.record(s_up)
            s_run.wait_event(up)
            init = (s0[b0:b1] if s0 is not None else None) if j == 0 else dev["sT"][b0:b1]
            wkv7_forward(*(dev[n][b0:b1, t0:t1] for n in _INPUTS), init, dev["y"][b0:b1, t0:t1],
                         dev["sT"][b0:b1], b1 - b0, t1 - t0, H, D, None, s_run)
            ran = torch.cuda.Event()
            ran.record(s_run)
            s_down.wait_event(ran)
            with torch.cuda.stream(s_down):
                y_host[b0:b1, t0:t1].copy_(dev["y"][b0:b1, t0:t1], non_blocking=True)
                if j == len(tb) - 2:
                    sT_host[b0:b1].copy_(dev["sT"][b0:b1], non_blocking=True)
    done = torch.cuda.Event()
    done.record(s_down)
    st.wait_event(done)


def forward_gated(r, w_log, k, v, a, b, r_k, g, s0=None, seq_offsets=None, want_state=True, stream=None):
    """Chunked prefill with the gated read-out z = (y / sqrt(D) + (sum r k r_k) v) * g.
    ``r_k`` is [H, D] fp32, ``g`` has the shape and dtype of ``r``.  Returns
    ``(z, sT)``."""
    import torch

    if seq_offsets is not None:
        T, H, D = r.shape
        B = seq_offsets.numel() - 1
    else:
        B, T, H, D = r.shape
    z = torch.empty_like(r)
    sT = torch.empty((B, H, D, D), dtype=torch.float32, device=r.device) if want_state else None
    wkv7_forward_gated(r, w_log, k, v, a, b, s0, r_k, g, z, sT, B, T, H, D, seq_offsets, stream)
    return z, sT


def forward_fused(r, w_log, k, v, a_lr, s0=None, seq_offsets=None, r_k=None, g=None, want_state=True, stream=None):
    """Chunked prefill with the fused prologue: ``k`` and ``v`` are the raw rows
    of the kv heads ([.., H_kv, D]), ``a_lr`` the in-context learning rate; the
    kernel forms kk, a = -kk, b = kk a_lr and k (1 - w + a_lr) itself.  With
    ``r_k`` and ``g`` the output is the gated read-out z.  Returns ``(y or z, sT)``."""
    import torch

    if seq_offsets is not None:
        T, H, D = r.shape
        B = seq_offsets.numel() - 1
    else:
        B, T, H, D = r.shape
    H_kv = k.shape[-2]
    out = torch.empty_like(r)
    sT = torch.empty((B, H, D, D), dtype=torch.float32, device=r.device) if want_state else None
    wkv7_forward_fused(r, w_log, k, v, a_lr, s0, r_k, g, out, sT, B, T, H, H_kv, D, seq_offsets, stream)
    return out, sT


def decode_step_fused(r, w_log, k, v, a_lr, state, r_k=None, g=None, out=None, stream=None):
    """One decoding step with the fused prologue (and the gated read-out when
    ``r_k`` and ``g`` are given), updating ``state`` in place.  ``k``, ``v`` are
    [B, H_kv, D].  Returns the output rows [B, H, D]."""
    import torch

    B, H, D = r.shape
    if out is None:
        out = torch.empty_like(r)
    wkv7_decode_step_fused(r, w_log, k, v, a_lr, state, r_k, g, out, state, B, H, k.shape[-2], D, stream)
    return out


def backward(r, w_log, k, v, a, b, dy, s0=None, dsT=None, seq_offsets=None, workspace=None, stream=None):
    """Gradient of <dy, y> + <dsT, sT> with respect to r, w_log, k, v, a, b and s0.
    Layouts as for ``forward``.  ``workspace`` (a device tensor of at least
    ``wkv7_backward_workspace_bytes`` bytes) is allocated when not given.
    Returns ``(dr, dw_log, dk, dv, da, db, ds0)``."""
    import torch

    if seq_offsets is not None:
        T, H, D = r.shape
        B = seq_offsets.numel() - 1
    else:
        B, T, H, D = r.shape
    if workspace is None:
        nbytes = wkv7_backward_workspace_bytes(B, T, H, D, seq_offsets is not None)
        workspace = torch.empty(nbytes // 4, dtype=torch.float32, device=r.device)
    grads = [torch.empty_like(x) for x in (r, w_log, k, v, a, b)]
    ds0 = torch.empty((B, H, D, D), dtype=torch.float32, device=r.device)
    wkv7_backward(r, w_log, k, v, a, b, s0, dy, dsT, grads[0], grads[1], grads[2], grads[3], grads[4], grads[5], ds0,
                  workspace, B, T, H, D, seq_offsets, stream)
    return tuple(grads) + (ds0,)


def decode_step(r, w_log, k, v, a, b, state, y=None, stream=None):
    """One decoding step, updating ``state`` ([B, H, D, D] fp32) in place.
    Returns y ([B, H, D])."""
    import torch

    B, H, D = r.shape
    if y is None:
        y = torch.empty_like(r)
    wkv7_decode_step(r, w_log, k, v, a, b, state, y, state, B, H, D, stream)
    return y


# ---------------------------------------------------------------- state-space layers
class _NoStream:
    """The current stream stays the current one."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_NO_STREAM = _NoStream()


def _outputs(like, stream, inputs):
    """The context in which outputs and workspaces of a call on ``stream`` are allocated:
    that stream's, so that the allocator hands their memory on only in its order.  The
    inputs are marked as used there."""
    if stream is None:
        return _NO_STREAM
    import torch

    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), like.device)
    for t in inputs:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


@functools.lru_cache(maxsize=256)
def _bytes(query, *sizes):
    """A workspace's size, asked of the library once per problem size."""
    return query(*sizes)


def _scratch(nbytes, like):
    """A workspace of at least ``nbytes`` bytes on the device of ``like``, or none."""
    return like.new_empty((nbytes + like.element_size() - 1) // like.element_size()) if nbytes else None


def _new(t):
    """A contiguous tensor of the shape, type and device of ``t``."""
    global _new
    import torch

    _new = functools.partial(torch.empty_like, memory_format=torch.contiguous_format)
    return _new(t)


def _rows(t, seq_offsets, inner):
    """(B, T) of [B, T, ..] or of packed [T, ..] rows with ``inner`` more dimensions."""
    want = inner + (1 if seq_offsets is not None else 2)
    if t.dim() != want:
        raise ValueError(f"expected {want} dimensions, not {t.dim()}")
    if seq_offsets is not None:
        return seq_offsets.numel() - 1, t.shape[0]
    return t.shape[0], t.shape[1]


def causal_conv(x, w, bias=None, s0=None, seq_offsets=None, act=None, want_state=True, stream=None):
    """Short causal convolution over tokens, one filter per channel, with an activation
    (``None`` or ``"silu"``).  ``x`` is [B, T, C], or packed [T, C] with int32
    ``seq_offsets`` [B+1] on the device; its rows may be slices of wider ones.  ``w`` is
    [C, W] fp32 with W of 2, 3 or 4, ``bias`` [C] fp32, ``s0`` [B, W-1, C] the rows before
    the first token.  Returns ``(y, sT)``: ``sT`` [B, W-1, C] (None when ``want_state`` is
    false) is the ``s0`` of the tokens that follow."""
    B, T = _rows(x, seq_offsets, 1)
    C, W = w.shape
    with _outputs(x, stream, (x, w, bias, s0, seq_offsets)):
        y = _new(x)
        sT = x.new_empty((B, W - 1, C)) if want_state else None
    wkv7_causal_conv(x, w, bias, s0, y, sT, B, T, C, W, seq_offsets, act, stream)
    return y, sT


def causal_conv_step(x, w, state, bias=None, act=None, y=None, stream=None):
    """One token per sequence of ``causal_conv``: ``x`` [B, C], ``state`` [B, W-1, C]
    updated in place.  Returns y ([B, C])."""
    C, W = w.shape
    if stream is not None:
        with _outputs(x, stream, (x, w, state, bias, y)):
            y = _new(x) if y is None else y
    elif y is None:
        y = _new(x)
    wkv7_causal_conv_step(x, w, bias, state, y, state, x.shape[0], C, W, act, stream)
    return y


def causal_conv_backward(x, w, dy, bias=None, s0=None, dsT=None, seq_offsets=None, act=None, workspace=None,
                         stream=None):
    """Gradient of <dy, y> + <dsT, sT> of ``causal_conv``.  Returns ``(dx, dw, dbias, ds0)``
    (``dbias`` is None without ``bias``)."""
    B, T = _rows(x, seq_offsets, 1)
    C, W = w.shape
    with _outputs(x, stream, (x, w, dy, bias, s0, dsT, seq_offsets, workspace)):
        if workspace is None:
            workspace = _scratch(_bytes(wkv7_causal_conv_backward_workspace_bytes, B, T, C, W, seq_offsets is not None), x)
        dx, dw = _new(x), _new(w)
        dbias = _new(bias) if bias is not None else None
        ds0 = x.new_empty((B, W - 1, C))
    wkv7_causal_conv_backward(x, w, bias, s0, dy, dsT, dx, dw, dbias, ds0, workspace, B, T, C, W, seq_offsets, act,
                              stream)
    return dx, dw, dbias, ds0


def selective_scan(x, dt, A, Bm, Cm, D=None, dt_bias=None, s0=None, seq_offsets=None, dt_softplus=True,
                   want_state=True, workspace=None, stream=None):
    """Selective state-space scan S_t = exp(A delta_t) S_{t-1} + delta_t x_t B_t^T,
    y_t = S_t C_t + D x_t with delta_t = softplus(dt_t + dt_bias).  ``x`` is [B, T, H, 64],
    ``dt`` [B, T, H], ``Bm`` and ``Cm`` [B, T, G, N] (N of 16, 32, 64 or 128; G divides H), or
    all packed along [T, ..] with int32 ``seq_offsets`` [B+1]; rows may be slices of wider
    ones.  ``A``, ``D`` and ``dt_bias`` are [H] fp32, ``s0`` [B, H, 64, N] fp32.
    ``workspace`` (a device tensor of at least ``wkv7_selective_scan_workspace_bytes``
    bytes) is allocated when not given.  Returns ``(y, sT)`` like ``forward``."""
    B, T = _rows(x, seq_offsets, 2)
    H, P = x.shape[-2:]
    G, N = Bm.shape[-2:]
    with _outputs(x, stream, (x, dt, A, Bm, Cm, D, dt_bias, s0, seq_offsets, workspace)):
        if workspace is None:
            workspace = _scratch(_bytes(wkv7_selective_scan_workspace_bytes, B, T, H, P, N, seq_offsets is not None), x)
        y = _new(x)
        sT = A.new_empty((B, H, P, N)) if want_state else None
    wkv7_selective_scan(x, dt, A, Bm, Cm, D, dt_bias, s0, y, sT, workspace, B, T, H, P, N, G, seq_offsets,
                        dt_softplus, stream)
    return y, sT


def selective_scan_step(x, dt, A, Bm, Cm, state, D=None, dt_bias=None, dt_softplus=True, y=None, stream=None):
    """One token per sequence of ``selective_scan``: ``x`` [B, H, 64], ``dt`` [B, H], ``Bm``
    and ``Cm`` [B, G, N], ``state`` [B, H, 64, N] fp32 updated in place.  Returns y
    ([B, H, 64])."""
    B, H, P = x.shape
    _, G, N = Bm.shape
    if stream is not None:
        with _outputs(x, stream, (x, dt, A, Bm, Cm, state, D, dt_bias, y)):
            y = _new(x) if y is None else y
    elif y is None:
        y = _new(x)
    wkv7_selective_scan_step(x, dt, A, Bm, Cm, D, dt_bias, state, y, state, B, H, P, N, G, dt_softplus, stream)
    return y


def selective_scan_backward(x, dt, A, Bm, Cm, dy, D=None, dt_bias=None, s0=None, dsT=None, seq_offsets=None,
                            dt_softplus=True, workspace=None, stream=None):
    """Gradient of <dy, y> + <dsT, sT> of ``selective_scan``.  Returns ``(dx, ddt, dA, dB, dC,
    dD, ddt_bias, ds0)`` (None for a parameter that was not given).
    ``wkv7_selective_scan_backward`` takes outputs of the caller, which may be slices of
    wider rows."""
    B, T = _rows(x, seq_offsets, 2)
    H, P = x.shape[-2:]
    G, N = Bm.shape[-2:]
    with _outputs(x, stream, (x, dt, A, Bm, Cm, dy, D, dt_bias, s0, dsT, seq_offsets, workspace)):
        if workspace is None:
            workspace = _scratch(
                _bytes(wkv7_selective_scan_backward_workspace_bytes, B, T, H, P, N, G, _code(x), seq_offsets is not None), x)
        dx, ddt, dA, dB, dC = (_new(t) for t in (x, dt, A, Bm, Cm))
        dD = _new(D) if D is not None else None
        dbias = _new(dt_bias) if dt_bias is not None else None
        ds0 = A.new_empty((B, H, P, N))
    wkv7_selective_scan_backward(x, dt, A, Bm, Cm, D, dt_bias, s0, dy, dsT, dx, ddt, dA, dB, dC, dD, dbias, ds0,
                                 workspace, B, T, H, P, N, G, seq_offsets, dt_softplus, stream)
    return dx, ddt, dA, dB, dC, dD, dbias, ds0


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, act=None, want_stats=False, workspace=None, stream=None):
    """Group norm with an activation (``None`` or ``"silu"``) over channels-last rows: ``x``
    [N, C] normalises the ``groups`` of every row (``groups`` = heads: the per-head norm of
    a recurrence's read-out), [N, L, C] takes the statistics over the L rows of a sample
    too.  ``weight`` and ``bias`` are [C] fp32.  Returns y, or ``(y, stats)`` with the
    ``stats`` [N, groups, 2] that ``group_norm_backward`` takes."""
    N, L, C = x.shape if x.dim() == 3 else (x.shape[0], 1, x.shape[-1])
    with _outputs(x, stream, (x, weight, bias, workspace)):
        if workspace is None:
            workspace = _scratch(_bytes(wkv7_group_norm_workspace_bytes, N, L, C, groups, _code(x)), x)
        y = _new(x)
        stats = _float32(x, (N, groups, 2)) if want_stats else None
    wkv7_group_norm(x, weight, bias, y, stats, workspace, N, L, C, groups, eps, act, stream)
    return (y, stats) if want_stats else y


def group_norm_backward(x, groups, stats, dy, weight=None, bias=None, act=None, workspace=None, stream=None):
    """Gradient of <dy, y> of ``group_norm``, from the statistics it returned.  Returns
    ``(dx, dweight, dbias)`` (None for a parameter that was not given)."""
    N, L, C = x.shape if x.dim() == 3 else (x.shape[0], 1, x.shape[-1])
    with _outputs(x, stream, (x, stats, dy, weight, bias, workspace)):
        if workspace is None:
            workspace = _scratch(_bytes(wkv7_group_norm_backward_workspace_bytes, N, L, C, groups, _code(x)), x)
        dx = _new(x)
        dw = _new(weight) if weight is not None else None
        db = _new(bias) if bias is not None else None
    wkv7_group_norm_backward(x, weight, bias, stats, dy, dx, dw, db, workspace, N, L, C, groups, act, stream)
    return dx, dw, db


def _float32(t, shape):
    import torch

    return torch.empty(shape, dtype=torch.float32, device=t.device)
