"""Refusals of the causal convolution, the selective scan and the group norm: bad arguments
are rejected on the host before anything is launched (no GPU needed), by the C entry
points with statuses and by the Python layer with exceptions.  And the fp64 references of
the GPU tests against autograd and differences."""
import pytest
import torch

import seq_reference as R


@pytest.fixture(scope="module")
def wk():
    import linear_recurrent_lm_wkv7_b200 as wk

    return wk


class Call:
    """A C entry point with valid arguments, some of them replaced."""

    def __init__(self, fn, names, ok):
        self.fn, self.names, self.ok = fn, names.split(), ok

    def __call__(self, **over):
        a = dict(self.ok)
        assert set(over) <= set(a), over
        a.update(over)
        return self.fn(*(a[n] for n in self.names))


MB = 1 << 20


def ptrs(*names):
    return {n: 0x10000000 + i * 64 * MB for i, n in enumerate(names)}


def conv_call(wk, step=False):
    lib = wk._lib()
    ok = ptrs("x", "w", "bias", "s0", "y", "sT") | dict(ldx=64, ldy=64, B=2, T=10, C=64, W=4, offs=None, act=1, io=1,
                                                        st=None)
    if step:
        return Call(lib.wkv7_causal_conv_step, "x ldx w bias s0 y ldy sT B C W act io st", ok)
    return Call(lib.wkv7_causal_conv, "x ldx w bias s0 y ldy sT B T C W offs act io st", ok)


@pytest.mark.parametrize("step", [False, True])
def test_conv_refusals(wk, step):
    call = conv_call(wk, step)
    assert call(B=0) == -1 and call(C=0) == -1 and call(W=0) == -1
    assert call(W=5) == -2 and call(W=1) == -2 and call(C=(1 << 20) + 1) == -2
    assert call(act=2) == -1 and call(io=5) == -1
    assert call(x=None) == -1 and call(w=None) == -1 and call(y=None) == -1
    assert call(ldx=63) == -1 and call(ldy=63) == -1 and call(ldx=1 << 31) == -1
    assert call(x=0x10000008) == -3 and call(sT=call.ok["sT"] + 4) == -3
    assert call(y=call.ok["x"] + 128) == -1  # y inside x
    assert call(y=call.ok["s0"]) == -1 and call(sT=call.ok["y"]) == -1
    assert call(sT=call.ok["s0"] + 64) == -1  # overlaps s0 without being it
    if step:
        assert call(sT=None) == -1
    else:
        assert call(T=-1) == -1 and call(T=(1 << 31) - 1, C=1 << 10) == -2
        # columns of one buffer may interleave, columns that overlap may not
        assert call(y=call.ok["x"] + 64, ldx=128, ldy=128) == -1


def test_a_state_in_place_lets_nothing_else_through(wk):
    """sT may be s0, and no other input even where that starts and ends with it: w, bias or x
    of the state's extent."""
    f32 = dict(io=0, C=64)
    call = conv_call(wk)
    for k, over in (("w", dict(B=2, W=2)), ("bias", dict(B=1, W=2)), ("x", dict(B=1, W=2, T=1)), ("x", dict(B=1, W=2, T=5))):
        assert call(**f32, **over, sT=call.ok[k], s0=None) == -1, k
        assert call(**f32, **over, sT=call.ok[k]) == -1, k
    step = conv_call(wk, True)
    for k, over in (("w", dict(B=2, W=2)), ("bias", dict(B=1, W=2)), ("x", dict(B=1, W=2))):
        assert step(**f32, **over, sT=step.ok[k]) == -1, k


def test_conv_backward_refusals(wk):
    lib = wk._lib()
    ok = ptrs("x", "w", "bias", "s0", "dy", "dsT", "dx", "dw", "db", "ds0", "ws") | dict(
        ldx=64, lddy=64, lddx=64, wsb=MB, B=2, T=10, C=64, W=4, offs=None, act=0, io=0, st=None)
    call = Call(lib.wkv7_causal_conv_backward,
                "x ldx w bias s0 dy lddy dsT dx lddx dw db ds0 ws wsb B T C W offs act io st", ok)
    need = wk.wkv7_causal_conv_backward_workspace_bytes(2, 10, 64, 4, False)
    assert need > 0 and call(wsb=need - 1) == -1
    assert call(dw=None) == -1 and call(dx=None) == -1 and call(ws=None) == -1 and call(W=7) == -2
    assert call(dx=ok["dy"]) == -1 and call(ds0=ok["s0"]) == -1 and call(db=ok["dw"] + 16) == -1
    assert call(ws=ok["x"]) == -1 and call(lddx=8) == -1 and call(dy=ok["dy"] + 2) == -3
    assert wk.wkv7_causal_conv_backward_workspace_bytes(0, 10, 64, 4, False) == 0


SCAN = "x ldx dt lddt A Bm ldb Cm ldc D bias s0 y ldy sT "


def scan_ok():
    return ptrs("x", "dt", "A", "Bm", "Cm", "D", "bias", "s0", "y", "sT", "ws") | dict(
        ldx=256, lddt=4, ldb=64, ldc=64, ldy=256, wsb=0, B=2, T=10, H=4, P=64, N=32, G=2, offs=None, sp=1, io=1, dtt=0,
        st=None)


@pytest.mark.parametrize("step", [False, True])
def test_scan_refusals(wk, step):
    lib, ok = wk._lib(), scan_ok()
    if step:
        call = Call(lib.wkv7_selective_scan_step, SCAN + "B H P N G sp io dtt st", ok)
    else:
        call = Call(lib.wkv7_selective_scan, SCAN + "ws wsb B T H P N G offs sp io dtt st", ok)
    assert call(B=0) == -1 and call(H=0) == -1 and call(G=3) == -1 and call(G=0) == -1
    assert call(P=32) == -2 and call(N=24) == -2 and call(N=256) == -2 and call(N=0) == -1
    assert call(io=3) == -1 and call(dtt=-1) == -1
    for k in ("x", "dt", "A", "Bm", "Cm", "y"):
        assert call(**{k: None}) == -1, k
    assert call(ldx=255) == -1 and call(ldb=63) == -1 and call(lddt=3) == -1
    assert call(ldx=260) == -3 and call(ldc=65) == -3  # bf16 rows off 16 bytes
    assert call(x=ok["x"] + 8) == -3 and call(dt=ok["dt"] + 2) == -3 and call(s0=ok["s0"] + 4) == -3
    assert call(y=ok["x"]) == -1 and call(sT=ok["x"]) == -1 and call(sT=ok["s0"] + 256) == -1
    if step:
        assert call(sT=None) == -1
    else:
        assert call(T=-1) == -1 and call(T=(1 << 31) - 1, H=1 << 12, ldx=1 << 18, ldy=1 << 18, lddt=1 << 12) == -2
        assert call(B=1 << 16, T=1 << 15) == -2  # 2^31 rows
        # a case that works in segments needs its workspace
        need = wk.wkv7_selective_scan_workspace_bytes(1, 20000, 4, 64, 32, False)
        assert need > 0 and call(B=1, T=20000, ws=None) == -1 and call(B=1, T=20000, wsb=need - 1) == -1
        assert call(B=1, T=20000, wsb=need, ws=ok["y"]) == -1
    # the decays of every chunk and head (5 x 64 + 4 floats), even in one segment
    assert wk.wkv7_selective_scan_workspace_bytes(1024, 64, 8, 64, 128, False) == 1024 * 8 * 324 * 4
    assert wk.wkv7_selective_scan_workspace_bytes(4, 0, 8, 64, 128, True) == 0
    assert wk.wkv7_selective_scan_workspace_bytes(1, 64, 8, 32, 128, False) == 0


def test_scan_backward_refusals(wk):
    lib = wk._lib()
    ok = scan_ok() | ptrs(*("p%d" % i for i in range(16)), "dy", "dsT", "dx", "ddt", "dA", "dB", "dC", "dD", "dbias",
                          "ds0", "bws") | dict(lddy=256, lddx=256, ldddt=4, lddb=64, lddc=64, wsb=64 * MB)
    call = Call(lib.wkv7_selective_scan_backward,
                "x ldx dt lddt A Bm ldb Cm ldc D bias s0 dy lddy dsT dx lddx ddt ldddt dA dB lddb dC lddc dD dbias ds0 "
                "bws wsb B T H P N G offs sp io dtt st", ok)
    need = wk.wkv7_selective_scan_backward_workspace_bytes(2, 10, 4, 64, 32, 2, 1, False)
    assert 0 < need <= 64 * MB and call(wsb=need - 1) == -1
    for k in ("dA", "dx", "ddt", "dB", "dC", "dy", "bws"):
        assert call(**{k: None}) == -1, k
    assert call(dx=ok["x"]) == -1 and call(dB=ok["dC"]) == -1 and call(ds0=ok["dsT"]) == -1
    assert call(lddx=264 - 4) == -3 and call(ldddt=3) == -1 and call(lddb=32) == -1
    assert wk.wkv7_selective_scan_backward_workspace_bytes(2, 10, 4, 64, 32, 3, 1, False) == 0
    # dx, dB and dC as columns of one buffer get past the overlap check (to the next refusal)
    cols = dict(dx=ok["dx"], dB=ok["dx"] + 512, dC=ok["dx"] + 512 + 128, lddx=384, lddb=384, lddc=384)
    assert call(**cols, dA=ok["dx"] + 256) == -1 and call(**(cols | dict(dC=ok["dx"] + 512 + 64))) == -1


def test_norm_refusals(wk):
    lib = wk._lib()
    ok = ptrs("x", "w", "b", "y", "stats", "ws", "dy", "dx", "dw", "db") | dict(
        ldx=64, ldy=64, lddy=64, lddx=64, wsb=0, N=3, L=1, C=64, G=4, eps=1e-5, act=1, io=1, st=None)
    call = Call(lib.wkv7_group_norm, "x ldx w b y ldy stats ws wsb N L C G eps act io st", ok)
    assert call(G=5) == -1 and call(G=0) == -1 and call(C=0) == -1 and call(N=-1) == -1 and call(L=-1) == -1
    assert call(eps=-1.0) == -1 and call(eps=float("nan")) == -1 and call(act=9) == -1 and call(io=2) == -1
    assert call(x=None) == -1 and call(y=None) == -1 and call(y=ok["x"]) == -1 and call(ldx=60) == -1
    assert call(x=ok["x"] + 2) == -3 and call(stats=ok["y"] + 16) == -1
    assert call(N=1 << 30) == -2 and call(N=1 << 29, C=64, G=4) == -2
    need = wk.wkv7_group_norm_workspace_bytes(3, 50, 64, 4, 1)
    assert need > 0 and call(L=50, ws=None) == -1 and call(L=50, wsb=need - 1) == -1
    assert wk.wkv7_group_norm_workspace_bytes(3, 1, 64, 4, 1) == 0
    back = Call(lib.wkv7_group_norm_backward, "x ldx w b stats dy lddy dx lddx dw db ws wsb N L C G act io st", ok)
    need = wk.wkv7_group_norm_backward_workspace_bytes(3, 1, 64, 4, 1)
    assert need > 0 and back(wsb=need - 1) == -1 and back(stats=None) == -1 and back(wsb=need, dx=ok["dy"]) == -1
    assert back(wsb=need, db=ok["dw"]) == -1 and back(G=7) == -1


@pytest.mark.parametrize("io,vec", [(0, 4), (1, 8)])
def test_norm_workspace_keeps_statistics_aligned(wk, io, vec):
    """The split form without statistics of the caller's keeps them, pairs of floats, at the
    end of the workspace: they begin on 16 bytes whatever the number of partial moments."""
    query = wk.wkv7_group_norm_workspace_bytes
    shapes = [(1, L, 960, 15) for L in (4104, 5000, 8192, 16000, 16384)]
    shapes += [(1, 16384, 480, 15), (1, 16384, 255, 15), (1, 16384, 255, 255), (3, 5001, 33, 11), (1, 1, 10007, 1)]
    shapes += [(N, L, Cg * G, G) for N in (1, 3, 7) for L in (2, 999, 4097, 11111) for G in (1, 3, 15, 41)
               for Cg in (1, 5, vec, 7 * vec, 64)]
    for N, L, C, G in shapes:
        n = query(N, L, C, G, io)
        assert n > 0 and (n - 8 * N * G) % 16 == 0, (N, L, C, G)


def test_python_refusals(wk):
    x = torch.zeros(2, 8, 16)
    w = torch.zeros(16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        wk.causal_conv(x, w)
    with pytest.raises(ValueError, match="dimensions"):
        wk.causal_conv(x[0], w)
    with pytest.raises(ValueError, match="CUDA"):
        wk.group_norm(x, 4)
    with pytest.raises(ValueError, match="act"):
        wk._binding._act("relu")
    ld = wk._binding._row_ld
    assert ld(torch.zeros(2, 8, 16), 2, 16, "x") == 16
    assert ld(torch.zeros(2, 8, 40)[..., 8:24], 2, 16, "x") == 40
    assert ld(torch.zeros(2, 8, 4, 64)[..., :2, :], 2, 128, "x") == 256
    assert ld(torch.zeros(2, 1, 40)[..., :16], 2, 16, "x") == 40  # one token per sequence
    assert ld(torch.zeros(1, 1, 5), 2, 5, "x") == 8 and ld(torch.zeros(2, 0, 5), 2, 5, "x") == 8
    with pytest.raises(ValueError, match="one stride"):
        ld(torch.zeros(2, 8, 16)[:, :5], 2, 16, "x")
    with pytest.raises(ValueError, match="contiguous"):
        ld(torch.zeros(2, 8, 32)[..., ::2], 2, 16, "x")
    with pytest.raises(ValueError, match="contiguous"):
        ld(torch.zeros(2, 8, 4, 80)[..., :64], 2, 256, "x")


@pytest.mark.parametrize("shape,lead,width", [((2 ** 32 + 8, 1), 1, 1), ((2, 2 ** 32 + 8, 1), 2, 1), ((2 ** 31, 1, 1), 2, 1),
                                              ((1, 2 ** 32 + 64), 1, 2 ** 32 + 64), ((2, 2, 2 ** 31), 2, 2 ** 31)])
def test_sizes_past_the_library_s_are_refused(wk, shape, lead, width):
    """The library counts in ints: a size that an int does not hold is refused, not cut to its
    low bits (2^32 + 8 rows would be 8)."""
    t = torch.empty(shape, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        wk._binding._rows(t, "x", t.dtype, t.shape, lead, width, t.get_device())


def test_steps_mark_every_tensor_for_another_stream(wk, monkeypatch):
    """A step on a stream that is given marks its inputs, the state and y as used there, also
    where y is the caller's."""
    marked = []
    monkeypatch.setattr(wk, "_outputs", lambda like, stream, inputs: marked.append((stream, inputs)) or wk._NO_STREAM)
    monkeypatch.setattr(wk, "wkv7_causal_conv_step", lambda *a: None)
    monkeypatch.setattr(wk, "wkv7_selective_scan_step", lambda *a: None)
    x, w, st, b, y = torch.zeros(2, 8), torch.zeros(8, 4), torch.zeros(2, 3, 8), torch.zeros(8), torch.zeros(2, 8)
    u, dt, A, B, S = torch.zeros(2, 4, 64), torch.zeros(2, 4), torch.zeros(4), torch.zeros(2, 1, 16), torch.zeros(2, 4, 64, 16)
    v = torch.zeros(2, 4, 64)
    for out, mine in ((y, [x, w, st, b, y]), (None, [x, w, st, b])):
        wk.causal_conv_step(x, w, st, bias=b, y=out, stream=7)
        stream, seen = marked.pop()
        assert stream == 7 and all(any(t is s for s in seen) for t in mine)
    for out, mine in ((v, [u, dt, A, B, S, v]), (None, [u, dt, A, B, S])):
        wk.selective_scan_step(u, dt, A, B, B, S, D=A, dt_bias=A, y=out, stream=7)
        stream, seen = marked.pop()
        assert stream == 7 and all(any(t is s for s in seen) for t in mine)
    assert wk.causal_conv_step(x, w, st, y=y) is y and not marked


# ---------------------------------------------------------------- the references themselves
def test_reference_scan_gradients():
    """The explicit gradients against autograd of the same recurrence."""
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    B, T, H, N, G = 2, 7, 4, 16, 2
    leaves = [t.requires_grad_(True) for t in (r(B, T, H, 64), r(B, T, H), -r(H).abs(), r(B, T, G, N), r(B, T, G, N),
                                               r(H), r(H), r(B, H, 64, N))]
    x, dt, A, Bm, Cm, D, bias, s0 = leaves
    dy, dsT = r(B, T, H, 64), r(B, H, 64, N)
    delta = torch.nn.functional.softplus(dt + bias)
    S, ys = s0, []
    for t in range(T):
        b, c = (m[:, t].repeat_interleave(H // G, 1) for m in (Bm, Cm))
        S = torch.exp(delta[:, t] * A)[..., None, None] * S + (delta[:, t][..., None] * x[:, t])[..., None] * b[:, :, None]
        ys.append((S * c[:, :, None]).sum(-1) + D[:, None] * x[:, t])
    y = torch.stack(ys, 1)
    want = torch.autograd.grad([y, S], leaves, [dy, dsT])
    out = R.scan(*leaves[:5], D, bias, s0, dy=dy, dsT=dsT)
    assert torch.allclose(out["y"], y, atol=1e-12) and torch.allclose(out["sT"], S, atol=1e-12)
    for k, v in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "ds0"), want):
        assert torch.allclose(out[k], v, rtol=1e-9, atol=1e-9), k
    big = R.scan(*leaves[:5], D, bias, s0, dy=dy, dsT=dsT, bound=True)
    assert all((big[k] >= out[k].abs() - 1e-9).all() for k in ("y", "sT", "dx", "ddt", "dA", "dB", "dC", "ds0"))


def test_reference_conv_and_norm_gradients():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    offs = torch.tensor([0, 5, 5, 6, 15], dtype=torch.int32)
    x, w, b, s0 = (t.requires_grad_(True) for t in (r(15, 6), r(6, 4), r(6), r(4, 3, 6)))
    dy, dsT = r(15, 6), r(4, 3, 6)
    ys, ends = [], []
    for n in range(4):
        full = torch.cat([s0[n], x[offs[n]:offs[n + 1]]])
        m = full.shape[0] - 3
        pre = b + sum(full[k:k + m] * w[:, k] for k in range(4))
        ys.append(pre * torch.sigmoid(pre))
        ends.append(full[m:])
    y, sT = torch.cat(ys), torch.stack(ends)
    want = torch.autograd.grad([y, sT], [x, w, b, s0], [dy, dsT])
    out = R.conv(x, w, b, s0, offs, "silu", dy, dsT)
    assert torch.allclose(out["y"], y) and torch.equal(out["sT"], sT)
    for k, v in zip(("dx", "dw", "dbias", "ds0"), want):
        assert torch.allclose(out[k], v, rtol=1e-9, atol=1e-12), k

    x, w, b = (t.requires_grad_(True) for t in (r(3, 4, 12), r(12), r(12)))
    dy = r(3, 4, 12)
    u = x.reshape(3, 4, 3, 4)
    h = (u - u.mean((1, 3), keepdim=True)) / (u.var((1, 3), keepdim=True, correction=0) + 1e-5) ** 0.5
    pre = h.reshape(x.shape) * w + b
    y = pre * torch.sigmoid(pre)
    want = torch.autograd.grad(y, [x, w, b], dy)
    out = R.norm(x, 3, w, b, activation="silu", dy=dy)
    assert torch.allclose(out["y"], y)
    for k, v in zip(("dx", "dweight", "dbias"), want):
        assert torch.allclose(out[k], v, rtol=1e-9, atol=1e-12), k
