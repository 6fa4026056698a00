"""Cases of the state-space operators and the group norm, for measuring them.

Three operators that stand beside the WKV recurrence:

* ``conv``: the short causal convolution over tokens, one filter per channel, with
  bias and SiLU (what a state-space layer applies to its x, B and C rows);
* ``scan``: the selective state-space scan with one decay per head and token,
  S_t = exp(A delta_t) S_{t-1} + delta_t x_t B_t^T,  y_t = S_t C_t + D x_t,
  delta = softplus(dt + dt_bias), on states of 64 x N per head, B and C shared by
  the heads of a group;
* ``norm``: group norm with an activation over channels-last rows.

Each is taken in up to three modes: ``prompt`` (whole sequences), ``step`` (one
token per sequence, the state updated in place) and ``train`` (forward, then every
gradient).  With ``own`` false, ``run`` computes the plain form in elementary torch
operations; with ``own`` true it calls the package.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
P = 64  # head size of the framework's recurrences
CHUNK = 64  # tokens per block of the plain scan


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one generated token for each of 256 sequences of a 2.9B-class layer (40 heads
        # of 64 channels and one group of B and C of 128 each): latency counts
        conv("conv_step_2p9b", "step", "bf16", B=256, T=1, C=2816, W=4),
        # a server's packed prompts in fp32, a channel count that fills no vector
        conv("conv_packed_f32", "prompt", "f32", B=16, T=16384, C=2307, W=3, packed=True, state=True, act="none"),
        # a training step of a 1.5B-class layer
        conv("conv_train_1p5b", "train", "bf16", B=4, T=1024, C=2304, W=4),
        # the smallest call: one generated token of one sequence
        scan("scan_step_one", "step", "bf16", B=1, T=1, H=32, N=128, G=1),
        # one generated token for each of 256 sequences: the states are the traffic
        scan("scan_step_2p9b", "step", "bf16", B=256, T=1, H=40, N=128, G=1),
        # the prompt of a 1.5B-class layer
        scan("scan_prompt_1p5b", "prompt", "bf16", B=4, T=1024, H=32, N=128, G=1),
        # one long document, continued from an earlier state
        scan("scan_long_2p9b", "prompt", "bf16", B=1, T=16384, H=40, N=128, G=1, state=True, slow=True),
        # packed prompts of uneven length in fp32, several groups of heads, a smaller state
        scan("scan_packed_f32", "prompt", "f32", B=9, T=5003, H=12, N=64, G=4, packed=True, state=True),
        # a training step of a 1.5B-class layer
        scan("scan_train_1p5b", "train", "bf16", B=4, T=1024, H=32, N=128, G=1),
        # the read-out of a 1.5B-class prompt, every token normalised per head
        norm("norm_rows_1p5b", "prompt", "bf16", N=4096, L=1, C=2048, G=32, act="silu"),
        # its training step
        norm("norm_train_1p5b", "train", "bf16", N=4096, L=1, C=2048, G=32, act="silu"),
        # statistics over whole sequences (an encoder's channels-last feature maps), odd sizes
        norm("norm_tokens_f32", "prompt", "f32", N=3, L=2111, C=960, G=15, act="silu"),
    ]


def conv(name, mode, io, B, T, C, W, packed=False, state=False, act="silu", bias=True):
    return dict(name=name, op="conv", mode=mode, io=io, B=B, T=T, C=C, W=W, packed=packed, state=state, act=act,
                bias=bias)


def scan(name, mode, io, B, T, H, N, G, packed=False, state=False, skip=True, slow=False):
    # slow: decays near one, so that the state remembers thousands of tokens
    return dict(name=name, op="scan", mode=mode, io=io, B=B, T=T, H=H, N=N, G=G, packed=packed, state=state,
                skip=skip, slow=slow)


def norm(name, mode, io, N, L, C, G, act):
    return dict(name=name, op="norm", mode=mode, io=io, N=N, L=L, C=C, G=G, act=act)


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    mode = rng.choice(["prompt", "step", "train"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        G = rng.choice([1, 2, 4, 15, 32, 40])
        C = G * _log(rng, 4, 2560 // G)
        if rng.random() < 0.6:  # a row per token
            N, L = _log(rng, 1, 8192), 1
        else:
            N = _log(rng, 1, 16)
            L = _log(rng, 2, max(2, 16384 // N))
        case = norm(None, "train" if mode == "train" else "prompt", io, N, L, C, G, rng.choice(["silu", "none"]))
    elif op == "conv":
        B = _log(rng, 1, 256) if mode == "step" else _log(rng, 1, 16)
        T = 1 if mode == "step" else _log(rng, 1, 16384 // B)
        packed = mode != "step" and rng.random() < 0.4
        C = _log(rng, 1, 2816) if rng.random() < 0.5 else 8 * _log(rng, 1, 352)
        case = conv(None, mode, io, B, T * B if packed else T, C, rng.choice([2, 3, 4]), packed,
                    rng.random() < 0.5, rng.choice(["silu", "none"]), rng.random() < 0.8)
    else:
        G = rng.choice([1, 1, 2, 4])
        H = G * _log(rng, 4 // G if mode == "train" else 1, 40 // G)
        N = rng.choice([16, 32, 64, 128])
        B = _log(rng, 1, 128) if mode == "step" else _log(rng, 1, 16)
        cap = 131072 // H if mode == "train" else min(16384, 524288 // H)
        T = 1 if mode == "step" else _log(rng, 1, max(1, cap // B))
        packed = mode != "step" and rng.random() < 0.4
        case = scan(None, mode, io, B, T * B if packed else T, H, N, G, packed, rng.random() < 0.5,
                    rng.random() < 0.8, rng.random() < 0.3)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs
class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
        self.h = torch.Generator().manual_seed(seed * 7919 + 17)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda")

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda")

    def lengths(self, B, total):
        """B lengths that add up to total: uneven, one of them empty and one a single
        token where there is room."""
        w = torch.rand(B, generator=self.h) + 0.1
        if B >= 4:
            w[1] = 0
        n = torch.floor(w / w.sum() * total).long().tolist()
        if B >= 4 and n[2] > 1:
            n[0] += n[2] - 1
            n[2] = 1
        n[-1] += total - sum(n)
        return n


def prepare(case, seed):
    """What a layer has in hand before the call.  Rows are column slices of wider
    buffers, as a projection or the convolution leaves them."""
    r = _Rand(seed)
    io = DT[case["io"]]
    s = {"case": case, "train": case["mode"] == "train", "step": case["mode"] == "step", "lens": None, "offs": None}
    if case["op"] == "norm":
        N, L, C = case["N"], case["L"], case["C"]
        shape = (N, C) if L == 1 else (N, L, C)
        s["x"] = (r.normal(*shape) * 1.5 + 0.3 * r.normal(C)).to(io)
        s["w"] = 1 + 0.1 * r.normal(C)
        s["b"] = 0.1 * r.normal(C)
        s["dy"] = r.normal(*shape).to(io) if s["train"] else None
        return s
    B, T = case["B"], case["T"]
    if case["packed"]:
        s["lens"] = r.lengths(B, T)
        offs = torch.zeros(B + 1, dtype=torch.int32)
        offs[1:] = torch.tensor(s["lens"]).cumsum(0)
        s["offs"] = offs.cuda()
    lead = (T,) if case["packed"] else (B,) if s["step"] else (B, T)
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        z = 64  # the columns of the projection that lie before the convolution's
        s["x"] = r.normal(*lead, z + (C + 7) // 8 * 8).to(io)[..., z:z + C]
        s["w"] = r.normal(C, W) / math.sqrt(W)
        s["b"] = 0.1 * r.normal(C) if case["bias"] else None
        s["s0"] = r.normal(B, W - 1, C).to(io) if case["state"] or s["step"] else None
        if s["train"]:
            s["dy"] = r.normal(*lead, C).to(io)
            s["dsT"] = r.normal(B, W - 1, C).to(io) if case["state"] else None
        return s
    H, N, G = case["H"], case["N"], case["G"]
    xbc = r.normal(*lead, H * P + 2 * G * N).to(io)
    s["x"] = xbc[..., :H * P].unflatten(-1, (H, P))
    s["Bm"] = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    s["Cm"] = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
    s["dt"] = r.normal(*lead, 64 + H).to(io)[..., 64:]
    s["A"] = -(1 + 15 * r.uniform(H))
    lo, hi = (1e-4, 1e-2) if case["slow"] else (1e-3, 1e-1)  # delta where dt is zero
    delta = torch.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * r.uniform(H))
    s["dt_bias"] = delta + torch.log(-torch.expm1(-delta))
    s["D"] = 1 + 0.1 * r.normal(H) if case["skip"] else None
    s["s0"] = 0.1 * r.normal(B, H, P, N) if case["state"] or s["step"] else None
    if s["train"]:
        s["dy"] = r.normal(*lead, H, P).to(io)
        s["dsT"] = 0.1 * r.normal(B, H, P, N) if case["state"] else None
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[op](state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[op](state)


def _own_conv(s):
    import linear_recurrent_lm_wkv7_b200 as wk

    act = s["case"]["act"]
    if s["step"]:
        y = wk.causal_conv_step(s["x"], s["w"], s["s0"], bias=s["b"], act=act)
        return y, s["s0"]
    y, sT = wk.causal_conv(s["x"], s["w"], bias=s["b"], s0=s["s0"], seq_offsets=s["offs"], act=act)
    if not s["train"]:
        return y, sT
    dx, dw, db, ds0 = wk.causal_conv_backward(s["x"], s["w"], s["dy"], bias=s["b"], s0=s["s0"], dsT=s["dsT"],
                                              seq_offsets=s["offs"], act=act)
    return (y, sT, dx, dw) + ((db,) if s["b"] is not None else ()) + ((ds0,) if s["s0"] is not None else ())


def _own_scan(s):
    import linear_recurrent_lm_wkv7_b200 as wk

    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    if s["step"]:
        y = wk.selective_scan_step(*args, s["s0"], D=s["D"], dt_bias=s["dt_bias"])
        return y, s["s0"]
    kw = dict(D=s["D"], dt_bias=s["dt_bias"], s0=s["s0"], seq_offsets=s["offs"])
    y, sT = wk.selective_scan(*args, **kw)
    if not s["train"]:
        return y, sT
    dx, ddt, dA, dB, dC, dD, dbias, ds0 = wk.selective_scan_backward(*args, s["dy"], dsT=s["dsT"], **kw)
    return (y, sT, dx, ddt, dA, dB, dC, dbias) + ((dD,) if s["D"] is not None else ()) + (
        (ds0,) if s["s0"] is not None else ())


def _own_norm(s):
    import linear_recurrent_lm_wkv7_b200 as wk

    G, act = s["case"]["G"], s["case"]["act"]
    if not s["train"]:
        return wk.group_norm(s["x"], G, s["w"], s["b"], act=act)
    y, stats = wk.group_norm(s["x"], G, s["w"], s["b"], act=act, want_stats=True)
    return (y,) + wk.group_norm_backward(s["x"], G, stats, s["dy"], s["w"], s["b"], act=act)


# ---------------------------------------------------------------- plain forms
def _leaves(train, *tensors):
    return [None if t is None else t.float().requires_grad_(True) if train else t.float() for t in tensors]


def _grads(outs, ups, leaves):
    pairs = [(o, u.float()) for o, u in zip(outs, ups) if u is not None]
    wrt = [t for t in leaves if t is not None]
    return list(torch.autograd.grad([o for o, _ in pairs], wrt, [u for _, u in pairs]))


def _sequences(s, n):
    """(sequence, first row, end row) of each packed sequence."""
    at = 0
    for i, m in enumerate(s["lens"]):
        yield i, at, at + m
        at += m


def _silu(x, act):
    return x / (1 + torch.exp(-x)) if act == "silu" else x


def _conv_rows(x, w, b, s0, act):
    """x [n, T, C] fp32 -> outputs [n, T, C] and the last W - 1 inputs."""
    n, T, C = x.shape
    W = w.shape[1]
    pad = x.new_zeros(n, W - 1, C) if s0 is None else s0
    xp = torch.cat([pad, x], 1)
    y = sum(xp[:, j:j + T] * w[:, j] for j in range(W))
    if b is not None:
        y = y + b
    return _silu(y, act), xp[:, T:]


def _plain_conv(s):
    c = s["case"]
    io = DT[c["io"]]
    if s["step"]:
        y, st = _conv_rows(s["x"].float()[:, None], s["w"], s["b"], s["s0"].float(), c["act"])
        s["s0"].copy_(st)
        return y[:, 0].to(io), s["s0"]
    x, w, b, s0 = leaves = _leaves(s["train"], s["x"], s["w"], s["b"], s["s0"])
    if c["packed"]:
        parts = [_conv_rows(x[None, i:j], w, b, None if s0 is None else s0[n:n + 1], c["act"])
                 for n, i, j in _sequences(s, c["B"])]
        y, sT = torch.cat([p[0][0] for p in parts]), torch.cat([p[1] for p in parts])
    else:
        y, sT = _conv_rows(x, w, b, s0, c["act"])
    if not s["train"]:
        return y.to(io), sT.to(io)
    g = _grads([y, sT], [s["dy"], s["dsT"]], leaves)
    out = [y.detach().to(io), sT.detach().to(io), g.pop(0).to(io), g.pop(0)]
    if b is not None:
        out.append(g.pop(0))
    if s0 is not None:
        out.append(g.pop(0).to(io))
    return tuple(out)


def _scan_rows(x, dt, A, Bm, Cm, D, bias, s0):
    """x [n, T, H, P] fp32 and so on -> y [n, T, H, P] and the last states [n, H, P, N].
    Blocks of up to CHUNK tokens: inside a block through the matrix of decays, from block to
    block through the state."""
    n, T, H, _ = x.shape
    G, N = Bm.shape[2:]
    S = x.new_zeros(n, H, P, N) if s0 is None else s0
    if T == 0:
        return torch.zeros_like(x), S
    delta = torch.nn.functional.softplus(dt + bias)
    m = min(CHUNK, T)
    K = -(-T // m)
    fill = K * m - T

    def cut(t):  # [n, T, ...] -> [n, K, m, ...], filled up with zeros (delta = 0 keeps the state)
        return torch.cat([t, t.new_zeros(n, fill, *t.shape[2:])], 1).unflatten(1, (K, m))

    xd = cut(x * delta[..., None])
    Bc = cut(Bm).repeat_interleave(H // G, 3)
    Cc = cut(Cm).repeat_interleave(H // G, 3)
    la = torch.cumsum(cut(delta.double() * A.double()), 2)  # log of the decay since the block's start
    gap = (la[:, :, :, None] - la[:, :, None]).permute(0, 1, 4, 2, 3)  # [n, K, H, t, s]
    keep = torch.ones(m, m, dtype=torch.bool, device=x.device).tril()
    M = torch.einsum("nkthi,nkshi->nkhts", Cc, Bc) * torch.exp(gap.masked_fill(~keep, -math.inf)).float()
    y = torch.einsum("nkhts,nkshp->nkthp", M, xd)
    add = torch.einsum("nkshp,nkshi->nkhpi", xd * torch.exp(la[:, :, -1:] - la).float()[..., None], Bc)
    decay = torch.exp(la[:, :, -1]).float()[..., None, None]
    starts = []
    for k in range(K):
        starts.append(S)
        S = decay[:, k] * S + add[:, k]
    y = y + torch.einsum("nkthi,nkhpi->nkthp", Cc, torch.stack(starts, 1)) * torch.exp(la).float()[..., None]
    y = y.flatten(1, 2)[:, :T]
    return (y if D is None else y + D[:, None] * x), S


def _plain_scan(s):
    c = s["case"]
    io = DT[c["io"]]
    if s["step"]:
        y, st = _scan_rows(*(t.float()[:, None] if t.dim() > 1 else t for t in
                             (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])), s["D"], s["dt_bias"], s["s0"])
        s["s0"].copy_(st)
        return y[:, 0].to(io), s["s0"]
    x, dt, A, Bm, Cm, bias, D, s0 = leaves = _leaves(s["train"], s["x"], s["dt"], s["A"], s["Bm"], s["Cm"],
                                                     s["dt_bias"], s["D"], s["s0"])
    if c["packed"]:
        parts = [_scan_rows(x[None, i:j], dt[None, i:j], A, Bm[None, i:j], Cm[None, i:j], D, bias,
                            None if s0 is None else s0[n:n + 1]) for n, i, j in _sequences(s, c["B"])]
        y, sT = torch.cat([p[0][0] for p in parts]), torch.cat([p[1] for p in parts])
    else:
        y, sT = _scan_rows(x, dt, A, Bm, Cm, D, bias, s0)
    if not s["train"]:
        return y.to(io), sT
    g = _grads([y, sT], [s["dy"], s["dsT"]], leaves)
    out = [y.detach().to(io), sT.detach()]
    for like in (io, io, None, io, io, None):  # dx, ddt, dA, dB, dC, ddt_bias
        t = g.pop(0)
        out.append(t if like is None else t.to(like))
    return tuple(out + g)


def _plain_norm(s):
    c = s["case"]
    io = DT[c["io"]]
    leaves = x, w, b = _leaves(s["train"], s["x"], s["w"], s["b"])
    u = x.reshape(c["N"], c["L"], c["G"], -1)
    d = u - u.mean((1, 3), keepdim=True)
    d = d / torch.sqrt((d * d).mean((1, 3), keepdim=True) + 1e-5)
    y = _silu(d.reshape(x.shape) * w + b, c["act"])
    if not s["train"]:
        return y.to(io)
    g = _grads([y], [s["dy"]], leaves)
    return y.detach().to(io), g[0].to(io), g[1], g[2]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["io"] == "bf16" else 4
    train = case["mode"] == "train"
    if case["op"] == "norm":
        n = case["N"] * case["L"] * case["C"]
        if train:  # x, dy in, y, dx out
            return {"bytes": 4 * n * e + 16 * case["C"], "flops": 22 * n}
        return {"bytes": 2 * n * e + 8 * case["C"], "flops": 9 * n}
    B = case["B"]
    rows = case["T"] if case["packed"] else B * case["T"]
    step = case["mode"] == "step"
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        st = B * (W - 1) * C * e * (2 if case["state"] or step else 1)  # the state in, the state out
        b = rows * C * e * 2 + C * (W + 1) * 4 + st
        f = rows * C * (2 * W + 4)
        if train:
            b += rows * C * e * 2 + C * (W + 1) * 4 + (st if case["state"] else 0)
            f += rows * C * (4 * W + 8)
        return {"bytes": b, "flops": f}
    H, N, G = case["H"], case["N"], case["G"]
    row = (2 * H * P + 2 * G * N + H) * e  # x, y, B, C, dt
    st = B * H * P * N * 4 * (2 if case["state"] or step else 1)
    b = rows * row + st + 12 * H
    f = rows * H * P * (5 * N + 2)  # decay, outer product and read-out of every state element
    if train:
        b += rows * (2 * H * P + 2 * G * N + H) * e + (st if case["state"] else 0) + 12 * H
        f += rows * H * P * (12 * N + 6)
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](case, f)


def _spans(case, f):
    """First and end row of every sequence in the rows flattened over the batch."""
    if case["packed"]:
        return [(i, j) for _, i, j in _sequences(f, case["B"])]
    return [(n * case["T"], (n + 1) * case["T"]) for n in range(case["B"])]


def _exact_conv(case, f):
    C, W, B = case["C"], case["W"], case["B"]
    x = f["x"].reshape(-1, C)
    spans = _spans(case, f)
    y, sT = torch.zeros_like(x), x.new_zeros(B, W - 1, C)
    dx, dw = torch.zeros_like(x), torch.zeros_like(f["w"])
    db, ds0 = x.new_zeros(C), x.new_zeros(B, W - 1, C)
    dy = f["dy"].reshape(-1, C) if f["train"] else None
    for n, (i, j) in enumerate(spans):
        head = x.new_zeros(W - 1, C) if f["s0"] is None else f["s0"][n]
        xp = torch.cat([head, x[i:j]])
        win = xp.unfold(0, W, 1) if j > i else x.new_zeros(0, C, W)  # [T, C, W]
        pre = (win * f["w"]).sum(-1)
        if f["b"] is not None:
            pre = pre + f["b"]
        sg = torch.sigmoid(pre)
        silu = case["act"] == "silu"
        y[i:j] = pre * sg if silu else pre
        sT[n] = xp[j - i:]
        if not f["train"]:
            continue
        g = dy[i:j] * (sg * (1 + pre * (1 - sg))) if silu else dy[i:j]
        db += g.sum(0)
        dw += (g[..., None] * win).sum(0)
        dxp = torch.zeros_like(xp)
        for k in range(W):
            dxp[k:k + j - i] += g * f["w"][:, k]
        if f["dsT"] is not None:
            dxp[j - i:] += f["dsT"][n]
        dx[i:j] = dxp[W - 1:]
        ds0[n] = dxp[:W - 1]
    shape = f["x"].shape
    if not f["train"]:
        return y.reshape(shape), sT
    return (y.reshape(shape), sT, dx.reshape(shape), dw) + ((db,) if f["b"] is not None else ()) + (
        (ds0,) if f["s0"] is not None else ())


def _exact_scan(case, f):
    """Token by token; sequences of a dense batch side by side.  The gradients walk
    back over the stored states."""
    H, N, G, B, T = (case[k] for k in "HNGBT")
    lead = f["x"].shape[:-2]
    if case["packed"]:
        groups = [(slice(n, n + 1), slice(i, j)) for n, i, j in _sequences(f, B)]
    else:
        groups = [(slice(0, B), slice(0, T))]

    def cut(t, span):  # -> [T, sequences, ...]
        if f["step"]:
            return t[None]
        return t[span][:, None] if case["packed"] else t[:, span].transpose(0, 1)

    def join(parts, tail):  # the inverse of cut, over all groups
        if f["step"]:
            return parts[0][0]
        if case["packed"]:
            return torch.cat([p[:, 0] for p in parts]).reshape(*lead, *tail)
        return parts[0].transpose(0, 1).reshape(*lead, *tail)

    ys, ends, dxs, ddts, dBs, dCs, ds0s = [], [], [], [], [], [], []
    A = f["A"]
    dA, dbias, dD = torch.zeros_like(A), torch.zeros_like(A), torch.zeros_like(A)
    rep = H // G
    for seqs, span in groups:
        x, raw, Bm, Cm = (cut(f[k], span) for k in ("x", "dt", "Bm", "Cm"))
        n = x.shape[1]
        raw = raw + f["dt_bias"]
        delta = torch.nn.functional.softplus(raw, threshold=700.0)
        a = torch.exp(delta * A)
        Bh, Ch = Bm.repeat_interleave(rep, 2), Cm.repeat_interleave(rep, 2)
        S = f["s0"][seqs].clone() if f["s0"] is not None else x.new_zeros(n, H, P, N)
        m = x.shape[0]
        kept = x.new_empty(m + 1, n, H, P, N) if f["train"] else None
        y = torch.empty_like(x)
        if kept is not None:
            kept[0] = S
        for t in range(m):
            S = a[t][..., None, None] * S
            S += (delta[t][..., None] * x[t])[..., None] * Bh[t][:, :, None]
            y[t] = (S @ Ch[t][..., None])[..., 0]
            if kept is not None:
                kept[t + 1] = S
        if f["D"] is not None:
            y += f["D"][:, None] * x
        ys.append(y)
        ends.append(S)
        if not f["train"]:
            continue
        dy = cut(f["dy"], span)
        dS = f["dsT"][seqs].clone() if f["dsT"] is not None else torch.zeros_like(S)
        du, ddel = torch.empty_like(x), torch.empty_like(delta)
        dBh, dCh = torch.empty_like(Bh), torch.empty_like(Ch)
        for t in range(m - 1, -1, -1):
            dCh[t] = (dy[t][:, :, None] @ kept[t + 1])[:, :, 0]
            dS += dy[t][..., None] * Ch[t][:, :, None]
            du[t] = (dS @ Bh[t][..., None])[..., 0]
            dBh[t] = ((delta[t][..., None] * x[t])[:, :, None] @ dS)[:, :, 0]
            ddel[t] = (dS * kept[t]).sum((-1, -2)) * a[t]  # of the logarithm of the decay
            dS *= a[t][..., None, None]
        dA += (ddel * delta).sum((0, 1))
        ddel = ddel * A + (du * x).sum(-1)
        ddt = ddel * torch.sigmoid(raw)
        dbias += ddt.sum((0, 1))
        dx = du * delta[..., None]
        if f["D"] is not None:
            dD += (dy * x).sum((0, 1, 3))
            dx = dx + f["D"][:, None] * dy
        dxs.append(dx)
        ddts.append(ddt)
        dBs.append(dBh.unflatten(2, (G, rep)).sum(3))
        dCs.append(dCh.unflatten(2, (G, rep)).sum(3))
        ds0s.append(dS)
        del kept
    y, sT = join(ys, (H, P)), torch.cat(ends)
    if not f["train"]:
        return y, sT
    return (y, sT, join(dxs, (H, P)), join(ddts, (H,)), dA, join(dBs, (G, N)), join(dCs, (G, N)), dbias) + (
        (dD,) if f["D"] is not None else ()) + ((torch.cat(ds0s),) if f["s0"] is not None else ())


def _exact_norm(case, f):
    N, L, C, G = case["N"], case["L"], case["C"], case["G"]
    x = f["x"].reshape(N, L, G, C // G)
    w, b = f["w"].reshape(G, -1), f["b"].reshape(G, -1)
    var, mean = torch.var_mean(x, (1, 3), correction=0, keepdim=True)
    rstd = (var + 1e-5) ** -0.5
    h = (x - mean) * rstd
    pre = h * w + b
    sg = torch.sigmoid(pre)
    silu = case["act"] == "silu"
    y = (pre * sg if silu else pre).reshape(f["x"].shape)
    if not f["train"]:
        return y
    g = f["dy"].reshape(x.shape)
    if silu:
        g = g * sg * (1 + pre * (1 - sg))
    gw = g * w
    dx = rstd * (gw - gw.mean((1, 3), keepdim=True) - h * (gw * h).mean((1, 3), keepdim=True))
    return y, dx.reshape(f["x"].shape), (g * h).sum((0, 1)).reshape(C), g.sum((0, 1)).reshape(C)
