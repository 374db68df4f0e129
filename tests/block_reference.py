"""The state-space block's operators in 64 bits, step by step, for the tests.

The backward passes are the formulas written out; tests/test_block_reference.py
checks them against finite differences.  Every function also takes `size=True`:
the same sums with every term's absolute value, which is what a rounding error
of each term is relative to."""
import torch

F64 = torch.float64


def sig(x):
    return 1 / (1 + torch.exp(-x))


def silu(x):
    return x * sig(x)


def dsilu(x):
    return sig(x) * (1 + x * (1 - sig(x)))


def each(p, rows):
    """Parameters [sets, ...] (or without sets) for every row."""
    return p.to(F64).repeat_interleave(rows // p.shape[0], 0)


def by_set(v, sets):
    return v.reshape(sets, -1, *v.shape[1:]).sum(1)


def row_lengths(lengths, rows, T):
    return [T] * rows if lengths is None else [int(n) for n in lengths]


def valid(lengths, rows, T, device):
    n = torch.tensor(row_lengths(lengths, rows, T), device=device)
    return (torch.arange(T, device=device)[None] < n[:, None]).unsqueeze(-1)


# ---- convolution ----------------------------------------------------------------

def conv(x, weight, bias=None, act=True, lengths=None, state=None, size=False):
    """(out, state_out, pre, inputs) with weight [S, K, D], bias [S, D]."""
    R, T, D = x.shape
    K = weight.shape[1]
    w = each(weight, R)
    on = valid(lengths, R, T, x.device)
    x = torch.where(on, x.to(F64), 0.0)
    before = torch.zeros(R, K - 1, D, dtype=F64, device=x.device) if state is None else state.to(F64)
    xs = torch.cat([before, x], 1)
    b = torch.zeros(R, D, dtype=F64, device=x.device) if bias is None else each(bias, R)
    pre = b[:, None].expand(R, T, D).clone()
    mag = pre.abs()
    for k in range(K):
        term = w[:, k, None] * xs[:, k:k + T]
        pre, mag = pre + term, mag + term.abs()
    out = torch.where(on, silu(pre) if act else pre, 0.0)
    # |d silu / d pre| <= 1.1
    err = torch.where(on, 1.1 * mag + out.abs(), 0.0)
    last = torch.stack([xs[r, n:n + K - 1] for r, n in enumerate(row_lengths(lengths, R, T))])
    return (err if size else out), last, pre, xs


def conv_backward(x, weight, dout, bias=None, act=True, lengths=None, state=None, dstate=None,
                  size=False):
    """(dx, dweight, dbias, dstate_in)."""
    R, T, D = x.shape
    S, K = weight.shape[:2]
    w = each(weight, R)
    on = valid(lengths, R, T, x.device)
    magp, _, pre, xs = conv(x, weight, bias, act, lengths, state, size=True)
    d = torch.where(on, dout.to(F64) * (dsilu(pre) if act else 1.0), 0.0)
    if size:
        # the slope's own error: |silu''| <= 1, so that of pre passes on with the factor 1
        d = torch.where(on, dout.to(F64).abs() * (1.1 + magp), 0.0)
        w, xs = w.abs(), xs.abs()
    dxs = torch.zeros(R, T + K - 1, D, dtype=F64, device=x.device)
    dw = []
    for k in range(K):
        dxs[:, k:k + T] += w[:, k, None] * d
        dw.append((d * xs[:, k:k + T]).sum(1))
    if dstate is not None:
        for r, n in enumerate(row_lengths(lengths, R, T)):
            e = dstate[r].to(F64)
            dxs[r, n:n + K - 1] += e.abs() if size else e
    return dxs[:, K - 1:], by_set(torch.stack(dw, 1), S), by_set(d.sum(1), S), dxs[:, :K - 1]


# ---- scan -----------------------------------------------------------------------

def steps(delta, bias, softplus):
    R = delta.shape[0]
    raw = delta.to(F64) + (0.0 if bias is None else each(bias, R)[:, None])
    return raw, (torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw)


def scan(u, delta, A, B, C, skip=None, z=None, bias=None, softplus=True, lengths=None, state=None,
         size=False):
    """(out, last state, all states [R, T+1, D, N], y) with A [S, D, N], skip and bias [S, D],
    B and C [R, T, G, N]."""
    R, T, D = u.shape
    N = A.shape[-1]
    on = valid(lengths, R, T, u.device)
    m = (lambda v: v.abs()) if size else (lambda v: v)
    raw, d = steps(delta, bias, softplus)
    d = torch.where(on, d, 0.0)
    Ar = each(A, R)
    u = torch.where(on, u.to(F64), 0.0)
    rep = D // B.shape[2]
    Bd = torch.where(on[..., None], m(B.to(F64)), 0.0).repeat_interleave(rep, 2)
    Cd = torch.where(on[..., None], m(C.to(F64)), 0.0).repeat_interleave(rep, 2)
    h = torch.zeros(R, D, N, dtype=F64, device=u.device) if state is None else m(state.to(F64))
    hs = [h]
    for t in range(T):
        h = torch.exp(d[:, t, :, None] * Ar) * h + m(d[:, t] * u[:, t])[..., None] * Bd[:, t]
        hs.append(h)
    hs = torch.stack(hs, 1)
    y = (hs[:, 1:] * Cd).sum(-1)
    if skip is not None:
        y = y + m(each(skip, R)[:, None] * u)
    out = y
    if z is not None:
        out = y * m(silu(z.to(F64)))
    return torch.where(on, out, 0.0), h, hs, torch.where(on, y, 0.0)


def scan_backward(u, delta, A, B, C, dout, skip=None, z=None, bias=None, softplus=True,
                  lengths=None, state=None, dstate=None, size=False):
    """Dict of gradients; B and C as in scan()."""
    R, T, D = u.shape
    S, _, N = A.shape
    G = B.shape[2]
    on = valid(lengths, R, T, u.device)
    m = (lambda v: v.abs()) if size else (lambda v: v)
    raw, d = steps(delta, bias, softplus)
    d = torch.where(on, d, 0.0)
    _, _, hs, y = scan(u, delta, A, B, C, skip, z, bias, softplus, lengths, state, size)
    Ar = each(A, R)
    u = m(torch.where(on, u.to(F64), 0.0))
    Bd = m(torch.where(on[..., None], B.to(F64), 0.0)).repeat_interleave(D // G, 2)
    Cd = m(torch.where(on[..., None], C.to(F64), 0.0)).repeat_interleave(D // G, 2)
    dout = m(torch.where(on, dout.to(F64), 0.0))
    out = {}
    dy = dout
    if z is not None:
        zz = torch.where(on, z.to(F64), 0.0)
        out["dz"] = dout * y * m(dsilu(zz))
        if size:
            out["dz"] = dout * y * 1.1
        dy = dout * m(silu(zz))
    sk = torch.zeros(R, 1, D, dtype=F64, device=u.device) if skip is None else m(each(skip, R)[:, None])
    g = torch.zeros(R, D, N, dtype=F64, device=u.device) if dstate is None else m(dstate.to(F64))
    slope = torch.where(on, sig(raw) if softplus else torch.ones_like(raw), 0.0)
    du, dr = torch.zeros_like(u), torch.zeros_like(u)
    dB, dC = torch.zeros(R, T, G, N, dtype=F64, device=u.device), torch.zeros(R, T, G, N, dtype=F64, device=u.device)
    dA = torch.zeros(R, D, N, dtype=F64, device=u.device)
    for t in reversed(range(T)):
        a = torch.exp(d[:, t, :, None] * Ar)
        g = g + Cd[:, t] * dy[:, t, :, None]
        dC[:, t] = (dy[:, t, :, None] * hs[:, t + 1]).reshape(R, G, D // G, N).sum(2)
        dB[:, t] = (g * (m(d[:, t]) * u[:, t])[..., None]).reshape(R, G, D // G, N).sum(2)
        gB = (g * Bd[:, t]).sum(-1)
        du[:, t] = gB * m(d[:, t]) + sk[:, 0] * dy[:, t]
        w = g * a * hs[:, t]
        dr[:, t] = ((w * m(Ar)).sum(-1) + gB * u[:, t]) * slope[:, t]
        dA = dA + w * m(d[:, t])[..., None]
        g = g * a
    out.update(du=du, ddelta=dr, dB=dB, dC=dC, dA=by_set(dA, S), dskip=by_set((dy * u).sum(1), S),
               ddelta_bias=by_set(dr.sum(1), S), dstate_in=g)
    return out


# ---- norms ------------------------------------------------------------------------

def norm(x, o=None, gate=None, w_post=None, scale=None, w_pre=None, eps=1e-6, gate_first=False):
    """(x_out, n_out or None); parameters [S, D]."""
    R = x.shape[0]
    x = x.to(F64)

    def rms(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)

    if o is not None:
        p = o.to(F64)
        act = 1.0 if gate is None else silu(gate.to(F64))
        if gate_first:
            p = p * act
        if w_post is not None:
            p = rms(p) * each(w_post, R)
        if not gate_first:
            p = p * act
        x = x + (p if scale is None else p * each(scale, R))
    return x, (None if w_pre is None else rms(x) * each(w_pre, R))


def norm_backward(y, dn=None, dx_out=None, o=None, gate=None, w_post=None, scale=None, w_pre=None,
                  eps=1e-6, gate_first=False):
    """Dict of gradients at the stored x_out = y."""
    R, D = y.shape
    y = y.to(F64)
    out = {}
    G = torch.zeros_like(y) if dx_out is None else dx_out.to(F64)
    if w_pre is not None:
        rn = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        e = dn.to(F64) * each(w_pre, R)
        G = G + rn * (e - y * rn * rn * (e * y).mean(1, keepdim=True))
        out["dw_pre"] = by_set(dn.to(F64) * y * rn, w_pre.shape[0])
    out["dx"] = G
    if o is None:
        return out
    o = o.to(F64)
    z = None if gate is None else gate.to(F64)
    act = torch.ones_like(o) if z is None else silu(z)
    v = o * act if gate_first else o
    wp = torch.ones_like(o) if w_post is None else each(w_post, R)
    sc = torch.ones_like(o) if scale is None else each(scale, R)
    after = torch.ones_like(o) if gate_first else act
    r = torch.ones(R, 1, dtype=F64, device=y.device) if w_post is None else \
        1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    p0 = v * r * wp
    if scale is not None:
        out["dscale"] = by_set(G * p0 * after, scale.shape[0])
    dp = G * sc
    dp0 = dp * after
    if w_post is not None:
        out["dw_post"] = by_set(dp0 * v * r, w_post.shape[0])
        e = dp0 * wp
        dv = r * (e - v * r * (e * v * r).mean(1, keepdim=True))
    else:
        dv = dp0
    out["do"] = dv * act if gate_first else dv
    if z is not None:
        out["dgate"] = (dv * o if gate_first else dp * p0) * dsilu(z)
    return out
