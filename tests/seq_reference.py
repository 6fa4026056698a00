"""fp64 references of the causal convolution, the selective scan and the group norm,
written token by token from their definitions, with explicit gradients.

Each returns its results as a dict.  ``bound=True`` gives, in the same places, the sums
of the absolute values of the terms that the result is a sum of: an error of e relative
to every term is at most e times that, which is what the tests' tolerances are
multiples of.  Inputs are CPU tensors of any type; packed batches come as offsets.
"""
import torch

P = 64


def spans(rows, offs, B, T):
    """(first row, end row) of every sequence in rows flattened over the batch."""
    if offs is not None:
        o = offs.tolist()
        return [(o[i], o[i + 1]) for i in range(len(o) - 1)]
    return [(n * T, (n + 1) * T) for n in range(B)]


def f64(t):
    return None if t is None else t.detach().cpu().double()


def act(u, name):
    return u * torch.sigmoid(u) if name == "silu" else u


def act_grad(u, name):
    if name != "silu":
        return torch.ones_like(u)
    s = torch.sigmoid(u)
    return s * (1 + u * (1 - s))


def conv(x, w, bias=None, s0=None, offs=None, activation=None, dy=None, dsT=None, bound=False):
    x, w, bias, s0, dy, dsT = (f64(t) for t in (x, w, bias, s0, dy, dsT))
    lead, C = x.shape[:-1], x.shape[-1]
    B, T = (len(offs) - 1, None) if offs is not None else lead
    W = w.shape[1]
    x = x.reshape(-1, C)
    y, sT = torch.zeros_like(x), x.new_zeros(B, W - 1, C)
    out = dict(dx=torch.zeros_like(x), dw=torch.zeros_like(w), dbias=x.new_zeros(C), ds0=x.new_zeros(B, W - 1, C))
    dy = dy.reshape(-1, C) if dy is not None else None
    ab = torch.abs if bound else (lambda t: t)
    for n, (i, j) in enumerate(spans(x, offs, B, T)):
        full = torch.cat([x.new_zeros(W - 1, C) if s0 is None else s0[n], x[i:j]])
        m = j - i
        pre = x.new_zeros(m, C) if bias is None else bias.expand(m, C).clone()
        size = pre.abs()
        for k in range(W):
            pre = pre + full[k:k + m] * w[:, k]
            size = size + (full[k:k + m] * w[:, k]).abs()
        # |act(u + d) - act(u)| <= 1.1 |d|
        y[i:j] = 1.1 * size + act(pre, activation).abs() if bound else act(pre, activation)
        sT[n] = ab(full[m:])
        if dy is None:
            continue
        g = dy[i:j] * act_grad(pre, activation)
        if bound:  # the slope of act' is at most 1/2
            g = g.abs() + 0.5 * dy[i:j].abs() * size + dy[i:j].abs()
        dfull = torch.zeros_like(full)
        for k in range(W):
            dfull[k:k + m] += g * ab(w[:, k])
            out["dw"][:, k] += (g * ab(full[k:k + m])).sum(0)
        if dsT is not None:
            dfull[m:] += ab(dsT[n])
        out["dbias"] += g.sum(0)
        out["dx"][i:j], out["ds0"][n] = dfull[W - 1:], dfull[:W - 1]
    out.update(y=y.reshape(*lead, C), sT=sT)
    out["dx"] = out["dx"].reshape(*lead, C)
    return out


def scan(x, dt, A, Bm, Cm, D=None, dt_bias=None, s0=None, offs=None, softplus=True, dy=None, dsT=None, bound=False):
    x, dt, A, Bm, Cm, D, dt_bias, s0, dy, dsT = (f64(t) for t in (x, dt, A, Bm, Cm, D, dt_bias, s0, dy, dsT))
    lead, (H, _) = x.shape[:-2], x.shape[-2:]
    G, N = Bm.shape[-2:]
    B, T = (len(offs) - 1, None) if offs is not None else lead
    x, dt = x.reshape(-1, H, P), dt.reshape(-1, H)
    Bm = Bm.reshape(-1, G, N).repeat_interleave(H // G, 1)
    Cm = Cm.reshape(-1, G, N).repeat_interleave(H // G, 1)
    raw = dt if dt_bias is None else dt + dt_bias
    delta = torch.nn.functional.softplus(raw, threshold=700.0) if softplus else raw
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    a = torch.exp(delta * A)
    if bound:
        x, Bm, Cm, A, delta = x.abs(), Bm.abs(), Cm.abs(), A.abs(), delta.abs()
        D, s0, dy, dsT = (None if t is None else t.abs() for t in (D, s0, dy, dsT))
    rows = x.shape[0]
    y, sT = torch.zeros_like(x), x.new_zeros(B, H, P, N)
    dx, ddt, dBh, dCh = torch.zeros_like(x), torch.zeros_like(dt), torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA, dD, ds0 = torch.zeros_like(A), torch.zeros_like(A), torch.zeros_like(sT)
    if dy is not None:
        dy = dy.reshape(-1, H, P)
    for n, (i, j) in enumerate(spans(x, offs, B, T)):
        S = [x.new_zeros(H, P, N) if s0 is None else s0[n]]
        for t in range(i, j):
            u = delta[t][:, None] * x[t]
            S.append(a[t][:, None, None] * S[-1] + u[:, :, None] * Bm[t][:, None])
            y[t] = torch.einsum("hpn,hn->hp", S[-1], Cm[t])
        sT[n] = S[-1]
        if dy is None:
            continue
        dS = x.new_zeros(H, P, N) if dsT is None else dsT[n]
        for t in range(j - 1, i - 1, -1):
            cur, prev = S[t - i + 1], S[t - i]
            dCh[t] = torch.einsum("hpn,hp->hn", cur, dy[t])
            dS = dS + dy[t][:, :, None] * Cm[t][:, None]
            du = torch.einsum("hpn,hn->hp", dS, Bm[t])
            dBh[t] = torch.einsum("hpn,hp->hn", dS, delta[t][:, None] * x[t])
            dla = (dS * prev).sum((1, 2)) * a[t]
            dA += dla * delta[t]
            ddt[t] = (dla * A + (du * x[t]).sum(-1)) * slope[t]
            dx[t] = delta[t][:, None] * du
            dS = a[t][:, None, None] * dS
        ds0[n] = dS
    if D is not None:
        y = y + D[:, None] * x
        if dy is not None:
            dx = dx + D[:, None] * dy
            dD = (dy * x).sum((0, 2))
    fold = lambda t: t.unflatten(1, (G, H // G)).sum(2).reshape(*lead, G, N)
    return dict(y=y.reshape(*lead, H, P), sT=sT, dx=dx.reshape(*lead, H, P), ddt=ddt.reshape(*lead, H), dA=dA,
                dB=fold(dBh), dC=fold(dCh), dD=dD, ddt_bias=ddt.sum(0), ds0=ds0, rows=rows)


def norm(x, groups, weight=None, bias=None, eps=1e-5, activation=None, dy=None, bound=False):
    x, weight, bias, dy = (f64(t) for t in (x, weight, bias, dy))
    N, C = x.shape[0], x.shape[-1]
    u = x.reshape(N, -1, groups, C // groups)
    w = (torch.ones(C, dtype=torch.float64) if weight is None else weight).reshape(groups, -1)
    b = (torch.zeros(C, dtype=torch.float64) if bias is None else bias).reshape(groups, -1)
    mean = u.mean((1, 3), keepdim=True)
    rstd = (((u - mean) ** 2).mean((1, 3), keepdim=True) + eps) ** -0.5
    h = (u - mean) * rstd
    size = (u.abs() + mean.abs()) * rstd + h.abs()  # of the terms of h
    pre = h * w + b
    psize = size * w.abs() + b.abs()
    out = dict(y=(1.1 * psize + act(pre, activation).abs() if bound else act(pre, activation)).reshape(x.shape),
               mean=mean.reshape(N, groups), rstd=rstd.reshape(N, groups))
    if dy is None:
        return out
    g = dy.reshape(u.shape) * act_grad(pre, activation)
    if bound:
        g = g.abs() + dy.reshape(u.shape).abs() * (1 + 0.5 * psize)
        h, w = size, w.abs()
    gw = g * w
    m1, m2 = gw.mean((1, 3), keepdim=True), (gw * h).mean((1, 3), keepdim=True)
    out["dx"] = (rstd * (gw + m1 + h * m2 if bound else gw - m1 - h * m2)).reshape(x.shape)
    out["dweight"], out["dbias"] = (g * h).sum((0, 1)).reshape(C), g.sum((0, 1)).reshape(C)
    return out
