"""Definitions in float64 (token after token, plain torch on the CPU) of the gated linear
recurrence and of the query/key norms with rotation, with the magnitudes that bound the
rounding errors of an fp32 evaluation. Shares no code with the library."""
import math

import torch

U32 = 2.0 ** -24                                            # half a step of fp32
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}  # of the type an output is stored in


def f64(t):
    return None if t is None else t.detach().cpu().double()


def gates(gate, form, scale):
    """a, s, da/dgate, ds/da in float64."""
    if form == "log":
        a, less, slope = gate.exp(), -torch.expm1(gate), gate.exp()
    elif form == "logit":
        a, less = torch.sigmoid(gate), torch.sigmoid(-gate)
        slope = a * less
    else:
        a, less, slope = gate, 1.0 - gate, torch.ones_like(gate)
    if scale == "complement":
        return a, less, slope, -torch.ones_like(a)
    if scale == "norm":
        s = (less * (1.0 + a)).sqrt()
        return a, s, slope, torch.where(s > 0, -a / s, 0.0)
    return a, torch.ones_like(a), slope, torch.zeros_like(a)


def recurrence(x, gate, h0=None, lengths=None, form="decay", scale="none"):
    """h, final_h and their magnitudes: the same walk over absolute values."""
    x, gate = f64(x), f64(gate)
    B, T, D = x.shape
    a, s, _, _ = gates(gate, form, scale)
    h = torch.zeros(B, D, dtype=torch.float64) if h0 is None else f64(h0).clone()
    m = h.abs()
    n = [T] * B if lengths is None else [min(max(int(v), 0), T) for v in lengths.cpu()]
    out, mag = torch.zeros_like(x), torch.zeros_like(x)
    for b in range(B):
        for t in range(n[b]):
            h[b] = a[b, t] * h[b] + s[b, t] * x[b, t]
            m[b] = a[b, t].abs() * m[b] + (s[b, t] * x[b, t]).abs()
            out[b, t], mag[b, t] = h[b], m[b]
    return out, h, mag, m


def recurrence_grads(x, gate, dh, h0=None, dfinal=None, lengths=None, form="decay", scale="none"):
    """{name: (gradient, magnitude)} of sum(dh h) + sum(dfinal final_h)."""
    h, _, hm, _ = recurrence(x, gate, h0, lengths, form, scale)
    x, gate, dh = f64(x), f64(gate), f64(dh)
    B, T, D = x.shape
    a, s, slope, ds = gates(gate, form, scale)
    start = torch.zeros(B, D, dtype=torch.float64) if h0 is None else f64(h0)
    mu = torch.zeros(B, D, dtype=torch.float64) if dfinal is None else f64(dfinal).clone()
    mm = mu.abs()
    n = [T] * B if lengths is None else [min(max(int(v), 0), T) for v in lengths.cpu()]
    dx, dg, dxm, dgm = (torch.zeros_like(x) for _ in range(4))
    for b in range(B):
        for t in range(n[b] - 1, -1, -1):
            before, bm = (h[b, t - 1], hm[b, t - 1]) if t else (start[b], start[b].abs())
            lam, lm = mu[b] + dh[b, t], mm[b] + dh[b, t].abs()
            dx[b, t], dxm[b, t] = s[b, t] * lam, s[b, t].abs() * lm
            dg[b, t] = lam * slope[b, t] * (before + x[b, t] * ds[b, t])
            dgm[b, t] = lm * slope[b, t].abs() * (bm + (x[b, t] * ds[b, t]).abs())
            mu[b], mm[b] = a[b, t] * lam, a[b, t].abs() * lm
    return {"dx": (dx, dxm), "dgate": (dg, dgm), "dh0": (mu, mm)}


def turn(y, positions, freqs, layout, amplitude, sign=1.0):
    """The rotation of y [B,T,H,W] by sign * position * freq, and the magnitude of each result."""
    rot = 2 * freqs.numel()
    ang = positions.double()[..., None] * freqs * sign
    c, s = amplitude * torch.cos(ang)[:, :, None], amplitude * torch.sin(ang)[:, :, None]
    i = torch.arange(rot // 2) if layout == "half" else torch.arange(0, rot, 2)
    j = i + (rot // 2 if layout == "half" else 1)
    out, mag = y.clone(), y.abs()
    out[..., i], out[..., j] = y[..., i] * c - y[..., j] * s, y[..., j] * c + y[..., i] * s
    both = abs(amplitude) * (y[..., i].abs() + y[..., j].abs())
    mag[..., i] = mag[..., j] = both
    return out, mag


def head_norm(x, w, norm, eps, scale, freqs, positions, layout, amplitude):
    """qk_norm on one tensor: the result and its magnitude."""
    x = f64(x)
    y = x
    if norm != "none":
        ss = x.square().sum(-1, keepdim=True) / (x.shape[-1] if norm == "rms" else 1)
        y = x * torch.where(ss + eps > 0, (ss + eps) ** -0.5, 0.0)
    y = y * scale * (1.0 if w is None else f64(w))
    return (y, y.abs()) if freqs is None else turn(y, positions, freqs, layout, amplitude)


def head_norm_grads(x, w, dout, norm, eps, scale, freqs, positions, layout, amplitude):
    """(dx, magnitude), (dw, magnitude) from the formulas; rows [B,T,H,W]."""
    x, g = f64(x), f64(dout)
    gm = g.abs()
    if freqs is not None:
        g, gm = turn(g, positions, freqs, layout, amplitude, -1.0)
    g, gm = g * scale, gm * abs(scale)
    if norm == "none":
        return (g, gm), None
    n = x.shape[-1] if norm == "rms" else 1
    ss = x.square().sum(-1, keepdim=True) / n + eps
    inv = torch.where(ss > 0, ss ** -0.5, 0.0)
    dw = (g * x * inv).sum((0, 1, 2)), (gm * (x * inv).abs()).sum((0, 1, 2))
    ww = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else f64(w)
    gw, gwm = g * ww, gm * ww.abs()
    dot, dotm = (gw * x).sum(-1, keepdim=True), (gwm * x.abs()).sum(-1, keepdim=True)
    k = inv * inv / n
    return (inv * (gw - x * k * dot), inv * (gwm + x.abs() * k * dotm)), dw


def close(got, want, mag, steps, what=""):
    """|got - want| <= half a step of got's type + steps fp32 roundings of the magnitude."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    g = f64(got)
    assert bool(torch.isfinite(g).all()), what
    limit = HALF_STEP[got.dtype] * (1 + 2.0 ** -8) * want.abs() + steps * U32 * mag + 1e-37
    bad = (g - want).abs() > limit
    if bool(bad.any()):
        k = int(torch.argmax(((g - want).abs() / limit).flatten()))
        raise AssertionError("%s: %d of %d off; worst got %.9g want %.9g limit %.3g" % (
            what, int(bad.sum()), bad.numel(), g.flatten()[k], want.flatten()[k], limit.flatten()[k]))


def positions_of(B, T, start=0):
    return (torch.arange(T) + start)[None].expand(B, T).contiguous()


def plain_freqs(rot, base=10000.0):
    return torch.tensor([math.pow(base, -2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
