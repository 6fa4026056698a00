"""GPU parity of the causal convolution, the selective scan and the group norm with the
fp64 references of seq_reference.py, through the public wrappers.

Tolerances, set before the first run.  An output of type t is rounded once: half a step,
eps(t) / 2 of its value.  What goes on inside is a sum of terms, each off by a relative e
(bound * e, the bound summing the terms' absolute values):
* fp32 arithmetic: a chain of m additions is off by m 2^-24 at most; m = 64 tokens of a
  chunk + N columns + the number of chunks (scan), W + 2 (convolution), and for sums over
  rows their number.  Exponentials and the sigmoid: 2^-21.
* the scan's fp32 values as bf16 planes: 2^-16 with two planes (outputs in bf16 alone),
  none with three.  Matrix units cut instead of rounding: 2^-23 an addition, so chains
  count twice.
"""
import pytest
import torch

import seq_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def wk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import linear_recurrent_lm_wkv7_b200 as wk

    return wk


def close(name, out, ref, bound, e):
    out, half = out.detach().cpu(), torch.finfo(out.dtype).eps / 2
    assert out.shape == ref.shape, (name, out.shape, ref.shape)
    assert torch.isfinite(out.float()).all(), f"{name}: not finite"
    tol = half * ref.abs() + e * (1 + half) * bound + 1e-30
    far = ((out.double() - ref).abs() / tol).max() if out.numel() else torch.tensor(0.0)
    assert far <= 1, f"{name}: {float(far):.2f} of the tolerance"


def offsets(lens):
    o = torch.zeros(len(lens) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(lens).cumsum(0)
    return o


def cuda(t):
    return None if t is None else t.cuda()


# ---------------------------------------------------------------- causal convolution
def conv_inputs(lead, B, C, W, io, seed, state=True, bias=True, wide=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    d = DT[io]
    x = r(*lead, C + wide).to(d)[..., wide // 2:wide // 2 + C] if wide else r(*lead, C).to(d)
    return dict(x=x, w=r(C, W), bias=r(C) if bias else None, s0=r(B, W - 1, C).to(d) if state else None,
                dy=r(*lead, C).to(d), dsT=r(B, W - 1, C).to(d) if state else None)


def wide_cuda(t, wide):
    """The same values as columns of a wider device buffer."""
    if not wide:
        return t.cuda()
    buf = torch.zeros(*t.shape[:-1], t.shape[-1] + wide, dtype=t.dtype, device="cuda")
    v = buf[..., wide // 2:wide // 2 + t.shape[-1]]
    v.copy_(t)
    return v


def check_conv(wk, inp, offs, activation, wide=0):
    x, w, bias, s0, dy, dsT = (inp[k] for k in ("x", "w", "bias", "s0", "dy", "dsT"))
    args = (x, w, bias, s0, offs, activation, dy, dsT)
    ref, bound = R.conv(*args), R.conv(*args, bound=True)
    xc, o = wide_cuda(x, wide), cuda(offs)
    y, sT = wk.causal_conv(xc, w.cuda(), cuda(bias), cuda(s0), o, activation)
    dx, dw, db, ds0 = wk.causal_conv_backward(xc, w.cuda(), dy.cuda(), cuda(bias), cuda(s0), cuda(dsT), o, activation)
    assert wk.wkv7_get_device_status() == 0
    e = (w.shape[1] + 2) * 2.0 ** -24 + 2.0 ** -21
    rows = x.numel() // x.shape[-1]
    close("y", y, ref["y"], bound["y"], e)
    assert torch.equal(sT.cpu().double(), ref["sT"])
    close("dx", dx, ref["dx"], bound["dx"], 2 * e)
    close("ds0", ds0, ref["ds0"], bound["ds0"], 2 * e)
    close("dw", dw, ref["dw"], bound["dw"], e + rows * 2.0 ** -24)
    if bias is not None:
        close("dbias", db, ref["dbias"], bound["dbias"], e + rows * 2.0 ** -24)
    else:
        assert db is None


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T,C", [(1, 8), (2, 5), (3, 64), (17, 24), (70, 33), (200, 40)])
def test_conv_dense(wk, io, W, T, C):
    check_conv(wk, conv_inputs((2, T), 2, C, W, io, seed=W * T + C), None, "silu" if C % 2 == 0 else None)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[5, 0, 1, 130, 2, 16, 0], [0, 0, 3], [64]])
def test_conv_packed(wk, io, lens):
    T = sum(lens)
    for W, C, state in ((4, 16, True), (3, 7, True), (2, 264, False)):
        check_conv(wk, conv_inputs((T,), len(lens), C, W, io, seed=W, state=state, bias=state), offsets(lens), "silu")


@pytest.mark.parametrize("wide", [8, 3])
def test_conv_rows_of_a_wider_buffer(wk, wide):
    """Row strides that keep vectors aligned, and ones that do not."""
    inp = conv_inputs((2, 33), 2, 48, 4, "f32", seed=wide)
    if wide == 3:  # the first column stays aligned, the stride does not
        buf = torch.zeros(2, 33, 51, device="cuda")
        xc = buf[..., :48]
        xc.copy_(inp["x"])
        ref, bound = R.conv(inp["x"], inp["w"], inp["bias"]), R.conv(inp["x"], inp["w"], inp["bias"], bound=True)
        y, _ = wk.causal_conv(xc, inp["w"].cuda(), inp["bias"].cuda())
        close("y", y, ref["y"], bound["y"], 6 * 2.0 ** -24)
    else:
        check_conv(wk, inp, None, "silu", wide=wide)


def test_conv_in_place_state_and_steps(wk):
    """A prompt in two calls with the state carried in place, then single tokens: the
    rows equal those of one call, bit for bit (the same sums in the same order)."""
    inp = conv_inputs((3, 41), 3, 40, 4, "bf16", seed=5)
    x, w, b, s0 = inp["x"].cuda(), inp["w"].cuda(), inp["bias"].cuda(), inp["s0"].cuda()
    y, sT = wk.causal_conv(x, w, b, s0, act="silu")
    st = s0.clone()
    parts = []
    for i, j in ((0, 2), (2, 30)):
        out = torch.empty(3, j - i, 40, dtype=x.dtype, device="cuda")
        wk.wkv7_causal_conv(x[:, i:j].contiguous(), w, b, st, out, st, 3, j - i, 40, 4, None, "silu")
        parts.append(out)
    for t in range(30, 41):
        parts.append(wk.causal_conv_step(x[:, t].contiguous(), w, st, bias=b, act="silu")[:, None])
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(st, sT)


# ---------------------------------------------------------------- selective scan
def scan_inputs(lead, B, H, N, G, io, seed, state=True, skip=True, decay=(1.0, 16.0), dt_shift=-3.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    d = DT[io]
    A = -(decay[0] + (decay[1] - decay[0]) * torch.rand(H, generator=g))
    return dict(x=r(*lead, H, 64).to(d), dt=r(*lead, H).to(d), A=A, Bm=r(*lead, G, N).to(d), Cm=r(*lead, G, N).to(d),
                D=r(H) if skip else None, dt_bias=dt_shift + r(H) if skip else None,
                s0=r(B, H, 64, N) if state else None, dy=r(*lead, H, 64).to(d),
                dsT=r(B, H, 64, N) if state else None)


def scan_e(inp, T):
    """(of outputs in the io type, of fp32 outputs): see the head of this file.  The terms
    of the gradients are products of two such sums, so those count twice again."""
    N = inp["Bm"].shape[-1]
    chain = 2 * (64 + N + T / 64) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22
    return chain + (2.0 ** -16 if inp["x"].dtype == torch.bfloat16 else 0.0), chain


def check_scan(wk, inp, offs=None, softplus=True, longest=None, grads=True):
    x, dt, A, Bm, Cm, D, bias, s0, dy, dsT = (inp[k] for k in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "s0", "dy",
                                                               "dsT"))
    args = (x, dt, A, Bm, Cm, D, bias, s0, offs, softplus) + ((dy, dsT) if grads else ())
    ref, bound = R.scan(*args), R.scan(*args, bound=True)
    T = longest or (x.shape[1] if offs is None else x.shape[0])
    e_io, e32 = scan_e(inp, T)
    dev = [cuda(t) for t in (x, dt, A, Bm, Cm)]
    kw = dict(D=cuda(D), dt_bias=cuda(bias), s0=cuda(s0), seq_offsets=cuda(offs), dt_softplus=softplus)
    y, sT = wk.selective_scan(*dev, **kw)
    assert wk.wkv7_get_device_status() == 0
    close("y", y, ref["y"], bound["y"], e_io)
    close("sT", sT, ref["sT"], bound["sT"], e32)
    if not grads:
        return
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "ds0")
    out = dict(zip(names, wk.selective_scan_backward(*dev, dy.cuda(), dsT=cuda(dsT), **kw)))
    assert wk.wkv7_get_device_status() == 0
    rows = x.shape[0] if offs is not None else x.shape[0] * x.shape[1]
    for k in names:
        if out[k] is None:
            assert k in ("dD", "ddt_bias") and D is None
            continue
        e = 2 * (e_io if k in ("dx", "dB", "dC") else e32)
        close(k, out[k], ref[k], bound[k], e + (rows * 2.0 ** -24 if k in ("dA", "dD", "ddt_bias") else 0))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130])
def test_scan_dense(wk, io, N, T):
    H, G = (4, 2) if N < 64 else (3, 1)
    check_scan(wk, scan_inputs((2, T), 2, H, N, G, io, seed=N + T))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_packed(wk, io):
    lens = [0, 5, 64, 1, 100, 0, 129, 0]
    inp = scan_inputs((sum(lens),), len(lens), 4, 32, 4, io, seed=7)
    check_scan(wk, inp, offsets(lens), longest=129)


@pytest.mark.parametrize("io,dt,N", [("f32", "bf16", 32), ("bf16", "f32", 32), ("bf16", "f32", 128)])
def test_scan_dt_of_another_type(wk, io, dt, N):
    """dt (and its gradient) in a type of its own, dense and packed."""
    lens = [100, 0, 150]
    for lead, B, offs in (((2, 130), 2, None), ((sum(lens),), 3, offsets(lens))):
        inp = scan_inputs(lead, B, 4, N, 2, io, seed=21)
        inp["dt"] = inp["dt"].to(DT[dt])
        check_scan(wk, inp, offs, longest=150)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_segments(wk, io):
    """Few heads and a long sequence: cut into segments, forwards and backwards, dense
    and packed; slow decays, so that states pass through many segments."""
    for packed in (False, True):
        lens = [700, 0, 1001]
        lead, B, offs = ((sum(lens),), 3, offsets(lens)) if packed else ((1, 1700), 1, None)
        assert wk.wkv7_selective_scan_workspace_bytes(B, 1700 if not packed else sum(lens), 2, 64, 16, packed) > 0
        inp = scan_inputs(lead, B, 2, 16, 1, io, seed=11, decay=(0.01, 0.1))
        check_scan(wk, inp, offs)


@pytest.mark.parametrize("T", [1, 127, 128, 129, 257, 400])
@pytest.mark.parametrize("H,G", [(3, 1), (4, 2)])
def test_scan_around_long_chunks(wk, T, H, G):
    """bf16 with 128 state columns works in chunks of 128 tokens."""
    check_scan(wk, scan_inputs((2, T), 2, H, 128, G, "bf16", seed=T + H))


def test_scan_long_chunks_segments(wk):
    lens = [1700, 0, 1, 1300]
    for lead, B, offs in (((1, 3000), 1, None), ((sum(lens),), 4, offsets(lens))):
        check_scan(wk, scan_inputs(lead, B, 2, 128, 1, "bf16", seed=12, decay=(0.01, 0.1)), offs)


@pytest.mark.parametrize("io,N", [("f32", 32), ("bf16", 32), ("bf16", 128)])
def test_scan_keeps_sequences_apart(wk, io, N):
    """Infinities and NaN in one packed sequence leave the others' bits alone."""
    lens = [70, 60, 130, 5]
    inp = scan_inputs((sum(lens),), 4, 4, N, 2, io, seed=N)
    d = {k: cuda(v) for k, v in inp.items()}
    offs = offsets(lens)
    bad = slice(int(offs[1]), int(offs[2]))
    ill = {k: v.clone() for k, v in d.items()}
    for k in ("x", "Bm", "Cm", "dt", "dy"):
        ill[k][bad] = float("nan")
        ill[k][bad.start] = float("inf")
    ill["s0"][1] = float("nan")
    outs = []
    for v in (d, ill):
        kw = dict(D=v["D"], dt_bias=v["dt_bias"], s0=v["s0"], seq_offsets=offs.cuda())
        y, sT = wk.selective_scan(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], **kw)
        g = wk.selective_scan_backward(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v["dy"], dsT=v["dsT"], **kw)
        outs.append((y, sT, g[0], g[1], g[3], g[4], g[7]))
    assert wk.wkv7_get_device_status() == 0
    rows = torch.ones(sum(lens), dtype=torch.bool)
    rows[bad] = False
    seqs = torch.tensor([True, False, True, True])
    for i, (a, b) in enumerate(zip(*outs)):
        keep = (seqs if i in (1, 6) else rows).cuda()
        assert torch.equal(a[keep], b[keep]), i


def test_scan_many_sequences(wk):
    """Hundreds of packed sequences of a few tokens, and their states."""
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 4, (300,), generator=g).tolist()
    for io, N in (("f32", 16), ("bf16", 128)):
        inp = scan_inputs((sum(lens),), 300, 2, N, 1, io, seed=1)
        check_scan(wk, inp, offsets(lens), longest=3)


@pytest.mark.parametrize("io,N", [("f32", 16), ("f32", 64), ("f32", 128), ("bf16", 16), ("bf16", 64), ("bf16", 128)])
def test_scan_long_sequences_keep_their_sums(wk, io, N):
    """Sequences of 8192 tokens that one block each carries from end to end, with decays near
    one.  All terms are positive, so that nothing cancels and what every step loses shows.
    Tolerance: K = 128 chunks, each multiplying the state by its decay (ex2: 2^-22) and adding
    its own sum (a rounding, 2^-24); that sum, from zero, of 4 steps of at most 6 products,
    each cut once (24 x 2^-23); delta 2^-20.  The tcgen05 kernels' chunks of 128 have 8 steps
    of 3.  dA is a sum of products of two states: twice that, and the sum over rows."""
    B, T, H = 4, 8192, 32
    g = torch.Generator(device="cuda").manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").abs().to(DT[io])
    x, Bm, Cm, dy = r(B, T, H, 64), r(B, T, 1, N), r(B, T, 1, N), r(B, T, H, 64)
    dt, A = r(B, T, H), -0.5 - torch.rand(H, generator=g, device="cuda")
    bias = torch.full((H,), -10.0, device="cuda")  # a decay of some e^-1 over the sequence
    s0, dsT = r(B, H, 64, N).float(), r(B, H, 64, N).float()
    # no segments: the workspace holds the chunks' decays alone
    assert wk.wkv7_selective_scan_workspace_bytes(B, T, H, 64, N, False) == B * T // 64 * H * 324 * 4
    kw = dict(dt_bias=bias, s0=s0)
    _, sT = wk.selective_scan(x, dt, A, Bm, Cm, **kw)
    grads = wk.selective_scan_backward(x, dt, A, Bm, Cm, dy, dsT=dsT, **kw)
    assert wk.wkv7_get_device_status() == 0

    delta = torch.nn.functional.softplus(dt.double() + bias.double())
    a = torch.exp(delta * A.double())
    keep = N == 16  # dA: 8.6 GB of states
    S, states = s0.double(), []
    for t in range(T):
        if keep:
            states.append(S)
        S = a[:, t, :, None, None] * S
        S += (delta[:, t, :, None] * x[:, t].double())[..., None] * Bm[:, t, :, None].double()
    dS, dA = dsT.double(), torch.zeros(H, dtype=torch.float64, device="cuda")
    for t in range(T - 1, -1, -1):
        dS = dS + dy[:, t].double()[..., None] * Cm[:, t, :, None].double()
        if keep:
            dA += ((dS * states.pop()).sum((2, 3)) * a[:, t] * delta[:, t]).sum(0)
        dS = a[:, t, :, None, None] * dS
    e = T // 64 * (2.0 ** -24 + 2.0 ** -22) + 24 * 2.0 ** -23 + 2.0 ** -20
    close("sT", sT, S.cpu(), S.cpu(), e)
    close("ds0", grads[7], dS.cpu(), dS.cpu(), e)
    if keep:
        close("dA", grads[2], dA.cpu(), dA.abs().cpu(), 2 * e + B * T * 2.0 ** -24)


@pytest.mark.parametrize("N", [16, 64, 128])
def test_scan_in_fp32_sums_like_fp32(wk, N):
    """A chunk of positive terms, where sums that are cut lose with one sign.  Each product of
    matrices sums up to N / 16 = 8 steps in fp32 (2^-24 each), a step's six products cut at its
    own size (2^-23): G or M 10 x 2^-24, the product with it (4 steps) 6 x 2^-24, the
    exponential 2^-22, delta and the factors' roundings 12 x 2^-24: 32 x 2^-24 = 2^-19 in all."""
    B, T, H = 2, 64, 2
    inp = scan_inputs((B, T), B, H, N, 1, "f32", seed=N, state=False, skip=False, decay=(0.1, 0.5))
    inp = {k: v if v is None or k == "A" else v.abs() for k, v in inp.items()}
    inp["dt"] *= 0.1
    names = ("x", "dt", "A", "Bm", "Cm")
    ref = R.scan(*(inp[k] for k in names), softplus=True, dy=inp["dy"])
    d = [cuda(inp[k]) for k in names]
    out = dict(zip(("y", "sT"), wk.selective_scan(*d)))
    grads = wk.selective_scan_backward(*d, inp["dy"].cuda())
    out.update(dx=grads[0], dB=grads[3], dC=grads[4])
    for k, v in out.items():
        close(k, v, ref[k], ref[k], 2.0 ** -19)


def test_calls_on_two_streams(wk):
    """The same kernels from two streams at once."""
    ins = []
    for seed in (1, 2):
        inp = scan_inputs((1, 3000), 1, 4, 128, 1, "bf16", seed=seed)
        ins.append({k: cuda(v) for k, v in inp.items()})
    call = lambda d, st=None: wk.selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], D=d["D"], dt_bias=d["dt_bias"],
                                                s0=d["s0"], stream=st)
    want = [call(d) for d in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[call(d, st) for _ in range(5)] for d, st in zip(ins, streams)]
    torch.cuda.synchronize()
    assert wk.wkv7_get_device_status() == 0
    for w, gs in zip(want, got):
        for y, sT in gs:
            assert torch.equal(y, w[0]) and torch.equal(sT, w[1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_without_options(wk, io):
    """No skip, bias, state or softplus; delta given as it is, zeros among it."""
    inp = scan_inputs((2, 70), 2, 2, 64, 1, io, seed=3, state=False, skip=False)
    inp["dt"] = inp["dt"].abs() * 0.1
    inp["dt"][:, 5:9] = 0
    check_scan(wk, inp, softplus=False)


def test_scan_strong_decays(wk):
    """delta A of -300 and more a token, and single tokens of almost none behind them:
    differences of large sums keep their bits."""
    inp = scan_inputs((1, 128), 1, 2, 16, 1, "f32", seed=4, decay=(60.0, 80.0), dt_shift=4.0)
    inp["dt"][:, 20:40] = -12.0
    inp["dt"][:, 70:75] = -20.0
    check_scan(wk, inp)


def test_scan_pad_tokens(wk):
    """dt = -inf leaves the state alone: the end state equals that of the sequence without
    those tokens."""
    inp = scan_inputs((1, 90), 1, 2, 32, 1, "f32", seed=9)
    keep = torch.ones(90, dtype=torch.bool)
    keep[10:14] = keep[60:70] = False
    inp["dt"][:, ~keep] = -float("inf")
    check_scan(wk, inp, grads=False)
    cut = {k: v[:, keep] if k in ("x", "dt", "Bm", "Cm") else v for k, v in inp.items()}
    ref, bound = (R.scan(*(cut[k] for k in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "s0")), bound=b) for b in (0, 1))
    _, sT = wk.selective_scan(*(inp[k].cuda() for k in ("x", "dt", "A", "Bm", "Cm")), D=inp["D"].cuda(),
                              dt_bias=inp["dt_bias"].cuda(), s0=inp["s0"].cuda())
    close("sT", sT, ref["sT"], bound["sT"], scan_e(inp, 90)[1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
def test_scan_steps_continue_a_prompt(wk, io, N):
    """A prompt, then single tokens with the state updated in place, against one scan."""
    inp = scan_inputs((3, 75), 3, 4, N, 2, io, seed=N)
    ref, bound = (R.scan(*(inp[k] for k in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "s0")), bound=b) for b in (0, 1))
    d = {k: cuda(v) for k, v in inp.items()}
    first = [d[k][:, :70].contiguous() if k != "A" else d[k] for k in ("x", "dt", "A", "Bm", "Cm")]
    y, st = wk.selective_scan(*first, D=d["D"], dt_bias=d["dt_bias"], s0=d["s0"])
    ys = [y]
    for t in range(70, 75):
        ys.append(wk.selective_scan_step(d["x"][:, t], d["dt"][:, t], d["A"], d["Bm"][:, t], d["Cm"][:, t], st,
                                         D=d["D"], dt_bias=d["dt_bias"])[:, None])
    e_io, e32 = scan_e(inp, 75)
    close("y", torch.cat(ys, 1), ref["y"], bound["y"], e_io)
    close("sT", st, ref["sT"], bound["sT"], e32)


def test_scan_state_in_place_and_rows_left_alone(wk):
    """sT over s0, and rows before the first and behind the last sequence."""
    inp = scan_inputs((80,), 2, 2, 16, 1, "bf16", seed=21)
    offs = torch.tensor([3, 40, 71], dtype=torch.int32)
    ref = R.scan(*(inp[k] for k in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "s0")), offs=offs)
    d = {k: cuda(v) for k, v in inp.items()}
    y = torch.full_like(d["x"], 7.0)
    st = d["s0"].clone()
    ws = torch.empty(max(16, wk.wkv7_selective_scan_workspace_bytes(2, 80, 2, 64, 16, True)), dtype=torch.uint8,
                     device="cuda")
    wk.wkv7_selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["dt_bias"], st, y, st, ws, 2, 80, 2, 64,
                           16, 1, offs.cuda())
    assert wk.wkv7_get_device_status() == 0
    assert (y[:3] == 7).all() and (y[71:] == 7).all()
    assert (y[3:71].cpu().double() - ref["y"][3:71]).abs().max() < 0.02 * ref["y"].abs().max()
    assert (st.cpu().double() - ref["sT"]).abs().max() < 1e-5 * ref["sT"].abs().max()
    g = {k: torch.full_like(d[s], 7.0) for k, s in (("dx", "x"), ("ddt", "dt"), ("dB", "Bm"), ("dC", "Cm"))}
    wsb = torch.empty(wk.wkv7_selective_scan_backward_workspace_bytes(2, 80, 2, 64, 16, 1, 1, True), dtype=torch.uint8,
                      device="cuda")
    dA = torch.empty(2, device="cuda")
    wk.wkv7_selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], None, None, None, d["dy"], None, g["dx"],
                                    g["ddt"], dA, g["dB"], g["dC"], None, None, None, wsb, 2, 80, 2, 64, 16, 1,
                                    offs.cuda())
    for k, v in g.items():
        assert (v[:3] == 7).all() and (v[71:] == 7).all(), k
        assert not (v[3:71] == 7).all(), k


def test_bad_offsets_are_reported(wk):
    """Offsets that leave the rows or run backwards: the sequences they bound are empty,
    nothing outside the tensors is touched, and the device status says so."""
    inp = scan_inputs((64,), 3, 2, 16, 1, "bf16", seed=2)
    d = {k: cuda(v) for k, v in inp.items()}
    offs = torch.tensor([0, 30, 20, 200], dtype=torch.int32).cuda()
    _, sT = wk.selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], s0=d["s0"], seq_offsets=offs)
    assert wk.wkv7_get_device_status() == -6
    assert torch.equal(sT[1:], d["s0"][1:])
    wk.selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], seq_offsets=offs)
    assert wk.wkv7_get_device_status() == -6
    x = torch.randn(64, 24, device="cuda")
    w = torch.randn(24, 4, device="cuda")
    wk.causal_conv(x, w, seq_offsets=offs)
    assert wk.wkv7_get_device_status() == -6
    wk.causal_conv_backward(x, w, x.clone(), seq_offsets=offs)
    assert wk.wkv7_get_device_status() == -6


@pytest.mark.parametrize("io,N", [("f32", 16), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("lens", [(0, 64, 10, 64), (0, 70, 64, 64), (0, -100, -100, 64), (0, 10, 64, 5)])
def test_bad_offsets_of_whole_sequences(wk, io, N, lens):
    """Every pair of offsets is looked at, also where sequences are not cut into segments: a bad
    one is reported, and its sequence's state (and state gradient) passes on."""
    T, B = 64, 3
    d = {k: cuda(v) for k, v in scan_inputs((T,), B, 2, N, 1, io, seed=2).items()}
    offs = torch.tensor(lens, dtype=torch.int32)
    bad = [n for n in range(B) if not 0 <= offs[n] <= offs[n + 1] <= T]
    assert bad
    kw = dict(s0=d["s0"], seq_offsets=offs.cuda())
    wk.wkv7_get_device_status()
    _, sT = wk.selective_scan(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], **kw)
    assert wk.wkv7_get_device_status() == -6
    ds0 = wk.selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], dsT=d["dsT"], **kw)[7]
    assert wk.wkv7_get_device_status() == -6
    for n in bad:
        assert torch.equal(sT[n], d["s0"][n]) and torch.equal(ds0[n], d["dsT"][n]), n


def test_bad_offsets_of_a_convolution_without_states(wk):
    """A bad pair between sequences that rows lead to is reported also where no state is wanted."""
    x, w = torch.randn(64, 24, device="cuda"), torch.randn(24, 4, device="cuda")
    for lens in ([0, 8, 4, 64], [0, 32, 16, 64], [0, 0, -3, 64]):
        offs = torch.tensor(lens, dtype=torch.int32).cuda()
        wk.wkv7_get_device_status()
        wk.causal_conv(x, w, seq_offsets=offs, want_state=False)
        assert wk.wkv7_get_device_status() == -6, lens
        ws = torch.empty(wk.wkv7_causal_conv_backward_workspace_bytes(3, 64, 24, 4, True), dtype=torch.uint8, device="cuda")
        wk.wkv7_causal_conv_backward(x, w, None, None, x.clone(), None, torch.empty_like(x), torch.empty_like(w), None, None,
                                     ws, 3, 64, 24, 4, offs)
        assert wk.wkv7_get_device_status() == -6, lens
    offs = offsets([5, 0, 59]).cuda()
    y, none = wk.causal_conv(x, w, seq_offsets=offs, want_state=False)
    assert none is None and torch.equal(y, wk.causal_conv(x, w, seq_offsets=offs)[0])
    assert wk.wkv7_get_device_status() == 0


def test_scan_gradient_against_differences(wk):
    """<dy, y> + <dsT, sT> of the kernels along a random direction in every input: central
    differences with step h have a relative error of h^2 and noise of e32 / h; with
    h = 2^-7 both are below 2^-9."""
    inp = scan_inputs((1, 100), 1, 4, 16, 2, "f32", seed=31)
    d = {k: cuda(v) for k, v in inp.items()}
    names = ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "s0")
    g = torch.Generator().manual_seed(1)
    way = {k: torch.randn(d[k].shape, generator=g).cuda() for k in names}
    grads = dict(zip(("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "s0"),
                     wk.selective_scan_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], D=d["D"],
                                                dt_bias=d["dt_bias"], s0=d["s0"], dsT=d["dsT"])))
    for k in names:
        h = 2.0 ** -7
        val = []
        for s in (h, -h):
            p = dict(d)
            p[k] = d[k] + s * way[k]
            y, sT = wk.selective_scan(p["x"], p["dt"], p["A"], p["Bm"], p["Cm"], D=p["D"], dt_bias=p["dt_bias"],
                                      s0=p["s0"])
            val.append((y.double() * d["dy"].double()).sum() + (sT.double() * d["dsT"].double()).sum())
        num = (val[0] - val[1]) / (2 * h)
        ana = (grads[k].double() * way[k].double()).sum()
        size = grads[k].double().norm() * way[k].double().norm()
        assert abs(num - ana) <= 2.0 ** -7 * max(abs(ana), size / way[k].numel() ** 0.5), k


# ---------------------------------------------------------------- group norm
def check_norm(wk, shape, groups, io, activation, affine=True, seed=0, shift=0.0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    C = shape[-1]
    x = (torch.randn(shape, generator=g) * scale + shift).to(DT[io])
    dy = torch.randn(shape, generator=g).to(DT[io])
    w = torch.randn(C, generator=g) if affine else None
    b = torch.randn(C, generator=g) if affine else None
    args = (x, groups, w, b, 1e-5, activation, dy)
    ref, bound = R.norm(*args), R.norm(*args, bound=True)
    y, stats = wk.group_norm(x.cuda(), groups, cuda(w), cuda(b), act=activation, want_stats=True)
    dx, dw, db = wk.group_norm_backward(x.cuda(), groups, stats, dy.cuda(), cuda(w), cuda(b), act=activation)
    n = x.numel() // (x.shape[0] * groups)
    rows = x.numel() // C
    e = 2.0 ** -21 + 2 * min(n, 2 * n ** 0.5 + 64) * 2.0 ** -24  # partial sums are short
    close("y", y, ref["y"], bound["y"], e)
    close("rstd", stats[..., 1], ref["rstd"], ref["rstd"], 2 * e)
    close("dx", dx, ref["dx"], bound["dx"], 3 * e)
    if affine:
        close("dweight", dw, ref["dweight"], bound["dweight"], 2 * e + rows * 2.0 ** -24)
        close("dbias", db, ref["dbias"], bound["dbias"], 2 * e + rows * 2.0 ** -24)
    else:
        assert dw is None and db is None


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C,groups", [(64, 1), (2048, 32), (40, 5), (33, 3), (7, 7), (24, 24), (520, 1), (2560, 1),
                                      (8200, 1), (1030, 1), (5, 1), (96, 2), (1600, 5)])
def test_norm_rows(wk, io, C, groups):
    for N, act in ((1, "silu"), (37, None), (300, "silu")):
        check_norm(wk, (N, C), groups, io, act, seed=C + N)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,L,C,groups", [(1, 2, 8, 1), (3, 17, 24, 3), (2, 300, 33, 11), (1, 1000, 64, 2),
                                          (5, 64, 4000, 4), (2, 3, 2600, 13)])
def test_norm_over_tokens(wk, io, N, L, C, groups):
    check_norm(wk, (N, L, C), groups, io, "silu", seed=L)
    check_norm(wk, (N, L, C), groups, io, None, affine=False, seed=L + 1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,L,C,groups", [(1, 16384, 960, 15), (1, 16000, 960, 15), (1, 5000, 960, 15),
                                          (1, 16384, 255, 15), (1, 12000, 255, 255), (3, 9001, 240, 240)])
def test_norm_joined_by_a_launch(wk, io, N, L, C, groups):
    """Few samples of many rows and groups: more moments than the blocks that write y join on
    the side, so a launch of its own joins them.  (Blocks' moments: splits x (groups of a tile
    + 1) x (tiles of a group + 1), above 8192 in fp32 for all of these.)  With and without
    statistics of the caller's, and the gradient."""
    check_norm(wk, (N, L, C), groups, io, "silu", seed=L + C)
    x = (torch.randn(N, L, C, generator=torch.Generator().manual_seed(C)) + 0.5).to(DT[io]).cuda()
    y, stats = wk.group_norm(x, groups, want_stats=True)
    assert torch.equal(wk.group_norm(x, groups), y) and torch.isfinite(stats).all()
    assert wk.wkv7_get_device_status() == 0


@pytest.mark.parametrize("shape", [(9, 128), (2, 50, 128)])
def test_norm_far_from_zero(wk, shape):
    """A mean of a thousand deviations: the squares are taken about the mean."""
    check_norm(wk, shape, 2, "f32", None, shift=1000.0)


def test_norm_many_samples(wk):
    """More samples than a grid dimension but the first holds."""
    x = torch.randn(70000, 2, 12, generator=torch.Generator().manual_seed(3))
    ref = R.norm(x, 3, activation="silu", dy=x)
    y, stats = wk.group_norm(x.cuda(), 3, act="silu", want_stats=True)
    dx, _, _ = wk.group_norm_backward(x.cuda(), 3, stats, x.cuda(), act="silu")
    assert float((y.cpu().double() - ref["y"]).norm() / ref["y"].norm()) < 2.0 ** -20
    assert float((dx.cpu().double() - ref["dx"]).norm() / ref["dx"].norm()) < 2.0 ** -18


def test_norm_keeps_samples_apart(wk):
    for shape in ((6, 64), (6, 40, 64)):
        x = torch.randn(shape, generator=torch.Generator().manual_seed(4)).cuda()
        y = wk.group_norm(x, 4, act="silu")
        ill = x.clone()
        ill[2] = float("nan")
        ill[4] = float("inf")
        z = wk.group_norm(ill, 4, act="silu")
        keep = [0, 1, 3, 5]
        assert torch.equal(y[keep], z[keep])


def test_conv_keeps_sequences_apart(wk):
    inp = conv_inputs((60,), 3, 24, 4, "bf16", seed=6)
    offs = offsets([20, 21, 19]).cuda()
    d = {k: cuda(v) for k, v in inp.items()}
    ill = {k: v.clone() for k, v in d.items()}
    ill["x"][20:41] = float("nan")
    ill["s0"][1] = float("inf")
    outs = [(*wk.causal_conv(v["x"], v["w"], v["bias"], v["s0"], offs, "silu"),
             *wk.causal_conv_backward(v["x"], v["w"], v["dy"], v["bias"], v["s0"], v["dsT"], offs, "silu")[::3])
            for v in (d, ill)]
    keep = torch.ones(60, dtype=torch.bool)
    keep[20:41] = False
    for i, (a, b) in enumerate(zip(*outs)):
        k = torch.tensor([True, False, True]).cuda() if i in (1, 3) else keep.cuda()
        assert torch.equal(a[k], b[k]), i


def test_norm_constant_rows(wk):
    x = torch.full((4, 64), 3.0, device="cuda")
    y, stats = wk.group_norm(x, 4, want_stats=True)
    assert (y == 0).all() and (stats[..., 0] == 3).all()
    assert torch.allclose(stats[..., 1], torch.full_like(stats[..., 1], 1e-5 ** -0.5))
    assert wk.group_norm(x[:0], 4).shape == (0, 64)
    dx, dw, db = wk.group_norm_backward(x[:0], 4, stats[:0], x[:0], torch.ones(64, device="cuda"),
                                        torch.zeros(64, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_silu_keeps_its_bits_far_out(wk):
    """SiLU and its derivative, relative to their own size, from -85 to 85: a convolution whose
    last tap is 1 and a norm without deviation hand the activation its argument as it is.
    u s(u): exp 2^-22, the sum 2^-24, the division 2^-22 (2 ulp), the product 2^-24, which is
    below 2^-20.5.  The derivative s (1 + u (1 - s)): s and 1 - s are off by 2^-21 of s and of 1,
    so 2^-20 of s (1 + |u|)."""
    u = torch.linspace(-85, 85, 8 * 4001, dtype=torch.float64).float()
    x = u.view(1, 4001, 8).cuda()
    w = torch.zeros(8, 4, device="cuda")
    w[:, 3] = 1
    s = torch.sigmoid(u.double())
    y, _ = wk.causal_conv(x, w, act="silu")
    dx, _, _, _ = wk.causal_conv_backward(x, w, torch.ones_like(x), act="silu")
    ref, slope = u.double() * s, s * (1 + u.double() * (1 - s))
    close("y", y.view(-1), ref, ref.abs(), 2.0 ** -20.5)
    # rows of one value: h = 0, and the bias is the argument
    z = wk.group_norm(torch.ones(1, u.numel(), device="cuda"), u.numel() // 8, None, u.cuda(), act="silu")
    close("z", z[0], ref, ref.abs(), 2.0 ** -20.5)
    close("dx", dx.view(-1), slope, s * (1 + u.double().abs()), 2.0 ** -20)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_silu_at_the_ends_of_the_range(wk, io):
    """Arguments far past where the exponential overflows or vanishes: 0 or the argument; +inf
    stays, NaN stays."""
    u = torch.tensor([-3e38, -1e30, -1e9, -1e4, -200.0, 200.0, 1e4, 1e9, 1e30, 3e38, float("inf"), float("nan")]).to(DT[io])
    want = torch.where(u < 0, torch.zeros_like(u), u)
    rows = u.view(-1, 1, 1).expand(-1, 1, 8).contiguous().cuda()
    w = torch.zeros(8, 4, device="cuda")
    w[:, 3] = 1
    y = wk.causal_conv(rows, w, act="silu")[0].cpu()
    assert all(torch.equal(y[:, 0, c].nan_to_num(7.0, 9.0), want.nan_to_num(7.0, 9.0)) for c in range(8))
    dx = wk.causal_conv_backward(rows[:10], w, torch.ones_like(rows[:10]), act="silu")[0].cpu()
    assert torch.equal(dx[:, 0, 0].float(), (u[:10] > 0).float())
    z = wk.group_norm(torch.ones(1, u.numel() * 8, dtype=DT[io], device="cuda"), u.numel(), None,
                      u.float().repeat_interleave(8).cuda(), act="silu").cpu().view(-1, 8)
    assert all(torch.equal(z[:, c].nan_to_num(7.0, 9.0), want.nan_to_num(7.0, 9.0)) for c in range(8))


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_layer(wk, io):
    """Convolution, scan and read-out norm as a layer runs them: the scan takes columns of
    the convolution's output, the backward of the scan writes into columns of one buffer
    that the convolution's backward takes; prompt and tokens against one pass."""
    B, T, H, N, G, W = 2, 90, 4, 32, 2, 4
    C = H * 64 + 2 * G * N
    d = DT[io]
    g = torch.Generator().manual_seed(17)
    r = lambda *s: torch.randn(*s, generator=g)
    u, dt = r(B, T, C).to(d), r(B, T, H).to(d)
    w, b, A, D, bias = r(C, W) * 0.5, r(C) * 0.1, -1 - 4 * torch.rand(H, generator=g), r(H), r(H) - 3
    nw, nb, dz = 1 + 0.1 * r(H * 64), 0.1 * r(H * 64), r(B * T, H * 64).to(d)
    cut = lambda t: (t[..., :H * 64].unflatten(-1, (H, 64)), t[..., H * 64:H * 64 + G * N].unflatten(-1, (G, N)),
                     t[..., H * 64 + G * N:].unflatten(-1, (G, N)))
    wc, bc, Ac, Dc, biasc, nwc, nbc = (t.cuda() for t in (w, b, A, D, bias, nw, nb))
    uc, dtc = u.cuda(), dt.cuda()

    def layer(u, dt, cs, ss):
        v, cs = wk.causal_conv(u, wc, bc, cs, act="silu")
        x, Bm, Cm = cut(v)
        y, ss = wk.selective_scan(x, dt, Ac, Bm, Cm, D=Dc, dt_bias=biasc, s0=ss)
        rows = y.flatten(0, 1).flatten(1)
        z, stats = wk.group_norm(rows, H, nwc, nbc, act="silu", want_stats=True)
        return z, v, rows, stats, cs, ss

    z, v, rows, stats, cT, sT = layer(uc, dtc, None, None)
    # forward against the references, each on the values it was given
    x, Bm, Cm = cut(v)
    ref = R.norm(rows, H, nw, nb, activation="silu", dy=dz)
    scale = 2.0 ** -7 if io == "bf16" else 2.0 ** -18
    near = lambda o, f: float((o.cpu().double() - f).norm() / f.norm()) < scale
    assert near(z, ref["y"])
    rs = R.scan(x, dt, A, Bm, Cm, D, bias, dy=ref["dx"].reshape(B, T, H, 64).to(d))
    assert near(rows, rs["y"].reshape(B * T, H * 64)) and near(sT, rs["sT"])
    rc = R.conv(u, w, b, activation="silu")
    assert near(v, rc["y"])
    # backward, without a copy between the operators
    drows, dnw, dnb = wk.group_norm_backward(rows, H, stats, dz.cuda(), nwc, nbc, act="silu")
    assert near(drows, ref["dx"]) and near(dnw, ref["dweight"])
    dv = torch.empty_like(v)
    dx, dB, dC = cut(dv)
    new = lambda t: torch.empty_like(t)
    ddt, dA, dD, dbias = torch.empty_like(dtc), new(Ac), new(Dc), new(biasc)
    ws = torch.empty(wk.wkv7_selective_scan_backward_workspace_bytes(B, T, H, 64, N, G, 0 if io == "f32" else 1, False),
                     dtype=torch.uint8, device="cuda")
    wk.wkv7_selective_scan_backward(x, dtc, Ac, Bm, Cm, Dc, biasc, None, drows.reshape(B, T, H, 64), None, dx, ddt, dA,
                                    dB, dC, dD, dbias, None, ws, B, T, H, 64, N, G)
    rs = R.scan(x, dt, A, Bm, Cm, D, bias, dy=drows.reshape(B, T, H, 64))
    for o, k in ((dx, "dx"), (ddt, "ddt"), (dB, "dB"), (dC, "dC"), (dA, "dA"), (dD, "dD"), (dbias, "ddt_bias")):
        assert near(o, rs[k]), k
    du, dw, db, _ = wk.causal_conv_backward(uc, wc, dv, bias=bc, act="silu")
    rc = R.conv(u, w, b, activation="silu", dy=dv)
    assert near(du, rc["dx"]) and near(dw, rc["dw"]) and near(db, rc["dbias"])
    # the same tokens as a prompt and then one by one
    z1, _, _, _, cs, ss = layer(uc[:, :80].contiguous(), dtc[:, :80].contiguous(), None, None)
    outs = [z1.reshape(B, 80, -1)]
    for t in range(80, T):
        x, Bm, Cm = cut(wk.causal_conv_step(uc[:, t], wc, cs, bias=bc, act="silu"))
        y = wk.selective_scan_step(x, dtc[:, t], Ac, Bm, Cm, ss, D=Dc, dt_bias=biasc)
        outs.append(wk.group_norm(y.flatten(1), H, nwc, nbc, act="silu")[:, None])
    # the norm passes errors of its input on, divided by the deviation of a group
    assert float((torch.cat(outs, 1).double() - z.reshape(B, T, -1).double()).norm() / z.double().norm()) < 4 * scale
    assert torch.equal(cs, cT) and float((ss - sT).norm() / sT.norm()) < 2.0 ** -16
    assert wk.wkv7_get_device_status() == 0


def test_graph_and_streams(wk):
    """Captured into a graph and replayed with new inputs; two graphs hold workspaces of
    their own; a call on a side stream."""
    inp = scan_inputs((1, 1500), 1, 2, 16, 1, "bf16", seed=8)
    d = {k: cuda(v) for k, v in inp.items()}
    call = lambda x: (wk.selective_scan(x, d["dt"], d["A"], d["Bm"], d["Cm"], D=d["D"], dt_bias=d["dt_bias"]),
                      wk.selective_scan_backward(x, d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], D=d["D"],
                                                 dt_bias=d["dt_bias"]))
    xs = [torch.randn_like(d["x"]) for _ in range(2)]
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    buf, graphs, outs = [torch.empty_like(xs[0]) for _ in range(2)], [], []
    for b in buf:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call(b))
        graphs.append(gr)
    flat = lambda o: list(o[0]) + list(o[1])
    for swap in (False, True):
        for b, x in zip(buf, xs[::-1] if swap else xs):
            b.copy_(x)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o, wnt in zip(outs, want[::-1] if swap else want):
            for a, b in zip(flat(o), flat(wnt)):
                assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, sT = wk.selective_scan(xs[0], d["dt"], d["A"], d["Bm"], d["Cm"], D=d["D"], dt_bias=d["dt_bias"], stream=side)
    side.synchronize()
    assert torch.equal(y, want[0][0][0]) and torch.equal(sT, want[0][0][1])


def test_steps_on_a_stream_keep_freed_inputs(wk):
    """An input that is freed behind a step on a busy stream is not handed out again before
    that stream is done with it, with y allocated and with y given."""
    side = torch.cuda.Stream()
    w, A = torch.randn(256, 4, device="cuda"), -torch.ones(4, device="cuda")
    x0, c0 = torch.randn(64, 256, device="cuda"), torch.randn(64, 3, 256, device="cuda")
    dt, b, s0 = (torch.randn(64, *s, device="cuda") for s in ((4,), (1, 16), (4, 64, 16)))

    def conv(x, st, y, stream):
        return wk.causal_conv_step(x, w, st, act="silu", y=y, stream=stream)

    def scan(x, st, y, stream):
        return wk.selective_scan_step(x.view(64, 4, 64), dt, A, b, b, st, y=None if y is None else y.view(64, 4, 64),
                                      stream=stream).view(64, 256)

    for call, state in ((conv, c0), (scan, s0)):
        want = call(x0, state.clone(), None, None)
        for given in (False, True):
            x, st, y = x0.clone(), state.clone(), torch.empty_like(x0) if given else None
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
            got = call(x, st, y, side)
            at = x.data_ptr()
            del x
            new = torch.full_like(x0, float("nan"))
            assert new.data_ptr() != at
            side.synchronize()
            assert torch.equal(got, want)


@pytest.mark.parametrize("io,N", [("bf16", 128), ("f32", 64)])
def test_calls_at_once(wk, io, N):
    """Calls of several kernels each, in turn on two streams and behind one another: every
    one gives the bits of a call alone."""
    ins = [{k: cuda(v) for k, v in scan_inputs((1, 1500), 1, 2, N, 1, io, seed=s).items()} for s in (1, 2)]

    def run(v, stream=None):
        kw = dict(D=v["D"], dt_bias=v["dt_bias"], s0=v["s0"], stream=stream)
        y = wk.selective_scan(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], **kw)
        g = wk.selective_scan_backward(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v["dy"], dsT=v["dsT"], **kw)
        rows = v["x"].reshape(1, 1500, -1)
        z = wk.causal_conv(rows, v["w"], act="silu", stream=stream)
        h = wk.causal_conv_backward(rows, v["w"], rows, act="silu", stream=stream)
        n = wk.group_norm(rows, 2, act="silu", stream=stream)
        return [t for o in (y, g, z, h, n) for t in o if t is not None]

    for s, v in enumerate(ins):
        v["w"] = torch.randn(128, 4, generator=torch.Generator().manual_seed(s)).cuda()
    want = [run(v) for v in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[run(v, st) for v, st in zip(ins, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for turn in got:
        for a, b in zip(turn, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert wk.wkv7_get_device_status() == 0


@pytest.mark.parametrize("N", [32, 128])
def test_offsets_past_32_bits(wk, N):
    """Rows so far apart that the last lie more than 2^31 elements behind the first."""
    T, H, ld = 600, 2, 1 << 22
    d = {k: cuda(v) for k, v in scan_inputs((T,), 1, H, N, 1, "bf16", seed=3).items()}
    buf = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    assert (T - 1) * ld > 1 << 31
    far = buf.as_strided((T, H, 64), (ld, 64, 1))
    far.copy_(d["x"])
    offs = offsets([T]).cuda()
    w = torch.randn(128, 4, generator=torch.Generator().manual_seed(1)).cuda()
    outs = []
    for x in (d["x"], far):
        rows = x.view(T, 128) if x is not far else buf.as_strided((T, 128), (ld, 1))
        kw = dict(s0=d["s0"][:1], seq_offsets=offs)
        out = list(wk.selective_scan(x, d["dt"], d["A"], d["Bm"], d["Cm"], **kw))
        out += wk.selective_scan_backward(x, d["dt"], d["A"], d["Bm"], d["Cm"], x, dsT=d["dsT"][:1], **kw)
        out += wk.causal_conv(rows, w, seq_offsets=offs, act="silu")
        out += wk.causal_conv_backward(rows, w, rows, seq_offsets=offs, act="silu")
        y, stats = wk.group_norm(rows, H, act="silu", want_stats=True)
        out += (y, stats, *wk.group_norm_backward(rows, H, stats, rows, act="silu"))
        outs.append([t.clone() for t in out if t is not None])
    assert wk.wkv7_get_device_status() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_empty_calls(wk):
    """No tokens: states pass on, gradients of parameters are zero."""
    s0 = torch.randn(2, 3, 24, device="cuda")
    w = torch.randn(24, 4, device="cuda")
    x = torch.empty(2, 0, 24, device="cuda")
    y, sT = wk.causal_conv(x, w, s0=s0)
    assert y.shape == x.shape and torch.equal(sT, s0)
    dx, dw, _, ds0 = wk.causal_conv_backward(x, w, x, s0=s0, dsT=s0)
    assert (dw == 0).all() and torch.equal(ds0, s0)
    S = torch.randn(2, 4, 64, 16, device="cuda")
    x, dt, b = (torch.empty(2, 0, *s, device="cuda") for s in ((4, 64), (4,), (1, 16)))
    A = -torch.ones(4, device="cuda")
    y, sT = wk.selective_scan(x, dt, A, b, b, s0=S)
    assert torch.equal(sT, S)
    out = wk.selective_scan_backward(x, dt, A, b, b, x, D=A, dt_bias=A, s0=S, dsT=S)
    assert all((out[k] == 0).all() for k in (2, 5, 6)) and torch.equal(out[7], S)
