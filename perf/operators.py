"""Cases that measure the operators around the delta-rule layer: the gated linear
recurrence, the norms of queries and keys with the position rotation, and the
rotation alone.

``run`` computes an operator in its plain form (elementary torch operations in 32
bits, angles in 64) or, where ``own`` is true, through the package's entry points.
``exact`` computes the same outputs in 64 bits straight from the definitions.

Gated linear recurrence, for every channel, with a_t from the gate:
    a = gate ("decay"), exp(gate) ("log"), 1 / (1 + exp(-gate)) ("logit");
    s = 1 ("none"), 1 - a ("complement"), sqrt(1 - a^2) ("norm");
    h_t = a_t h_{t-1} + s_t x_t.
Norms with rotation, for every token and head:
    y = scale w x / sqrt(mean x^2 + eps) ("rms") or scale x / sqrt(sum x^2 + eps) ("l2"),
    then (y_i, y_j) -> m (y_i cos - y_j sin, y_j cos + y_i sin) at the angle
    position * freq_i, where (i, j) are (i, i + rot / 2) ("half") or (2 i, 2 i + 1)
    ("interleaved") of the first rot features.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def _recurrence(name, mode, B, T, D, dtype, gate_dtype, gate, scale, docs=0, ragged=False, h0=True):
    return {"name": name, "op": "recurrence", "mode": mode, "B": B, "T": T, "D": D, "dtype": dtype,
            "gate_dtype": gate_dtype, "gate": gate, "scale": scale, "docs": docs, "ragged": ragged, "h0": h0}


def _heads(name, op, mode, B, T, Hq, Hk, width, dtype, norm, layout, rot, scaling, start=0):
    return {"name": name, "op": op, "mode": mode, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "width": width,
            "dtype": dtype, "norm": norm, "layout": layout, "rot": rot, "scaling": scaling, "start": start}


def listed():
    return [
        # one decode token of 256 sequences, the gate as a logit: latency counts
        _recurrence("recurrence step", "step", 256, 1, 2048, "bf16", "bf16", "logit", "complement"),
        # the forward of the 1.3B-shaped layer's width, batch and length, packed documents
        _recurrence("recurrence forward", "forward", 8, 4096, 2048, "bf16", "bf16", "log", "norm", docs=1024),
        # one long sequence: few channels, so the work has to be split over the tokens
        _recurrence("recurrence long", "forward", 1, 32768, 2048, "bf16", "fp32", "log", "none", h0=False),
        # a training step (forward and gradients) of the 340M-shaped layer
        _recurrence("recurrence train", "train", 8, 2048, 1024, "bf16", "bf16", "logit", "complement", docs=512),
        # a training step in fp32, odd sizes, sequences of different lengths
        _recurrence("recurrence train odd", "train", 3, 1777, 1001, "fp32", "fp32", "decay", "none", ragged=True),
        # queries and keys of the 1.3B-shaped layer, from one fused projection, as the delta rule wants them
        _heads("qk norm forward", "qk_norm", "forward", 8, 4096, 16, 16, 128, "bf16", "l2", "half", 128, "none"),
        # one decode token of 256 sequences, at far positions
        _heads("qk norm decode", "qk_norm", "forward", 256, 1, 16, 16, 128, "bf16", "rms", "half", 128, "none", 30000),
        # a training step with shared key heads, norm weights and a rotated part of the head
        _heads("qk norm train", "qk_norm", "train", 8, 2048, 16, 4, 128, "bf16", "rms", "half", 64, "none"),
        # fp32, odd length, 64 features, neighbouring pairs
        _heads("qk norm train odd", "qk_norm", "train", 3, 517, 5, 5, 64, "fp32", "l2", "interleaved", 32, "none"),
        # keys of a long context, frequencies scaled for eight times the trained length
        _heads("rotation long", "rope", "forward", 1, 32768, 16, 0, 128, "bf16", "none", "half", 128, "yarn", 100000),
        # one decode token of 256 sequences, part of the head, neighbouring pairs
        _heads("rotation decode", "rope", "forward", 256, 1, 16, 0, 128, "bf16", "none", "interleaved", 64, "linear", 5000),
        # the rotation and its gradient in fp32, odd sizes
        _heads("rotation train", "rope", "train", 3, 1021, 7, 0, 64, "fp32", "none", "interleaved", 64, "none"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """A case of the same ranges: up to the largest listed case's elements, odd sizes among them."""
    op = rng.choice(["recurrence", "recurrence", "qk_norm", "rope"])
    if op == "recurrence":
        mode = rng.choice(["forward", "train", "step"])
        dtype, gate_dtype = rng.choice([("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
        D = _log_int(rng, 64, 4096)
        D = D // 8 * 8 if rng.random() < 0.7 else D
        if mode == "step":
            B, T = _log_int(rng, 1, 512), 1
        else:
            T = _log_int(rng, 16, 32768)
            B = _log_int(rng, 1, 16)
            B = max(1, min(B, (16 << 20) // (T * D)))
            T = min(T, (16 << 20) // (B * D))
        gate = rng.choice(["decay", "log", "logit"])
        scale = rng.choice(["none", "complement"] if gate == "decay" else ["none", "complement", "norm"])
        c = _recurrence("", mode, B, T, D, dtype, gate_dtype, gate, scale,
                        docs=rng.choice([0, 0, 300]) if mode != "step" else 0,
                        ragged=mode != "step" and rng.random() < 0.3, h0=rng.random() < 0.7)
    else:
        T = rng.choice([1, _log_int(rng, 2, 16384)])
        B = _log_int(rng, 1, 256 if T == 1 else 8)
        width = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 4, 5, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        T = max(1, min(T, (16 << 20) // (B * (Hq + Hk) * width)))
        layout = rng.choice(["half", "interleaved"])
        rot = rng.choice([width, width // 2, 32])
        c = _heads("", op, rng.choice(["forward", "train"]), B, T, Hq, Hk if op == "qk_norm" else 0, width,
                   rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["l2", "rms"]) if op == "qk_norm" else "none",
                   layout, rot, rng.choice(["none", "linear", "yarn"]), rng.choice([0, rng.randrange(200000)]))
    del c["name"]
    return c


def _frequencies(rot, scaling):
    """The rotation's frequencies in 64 bits and the factor on its rotated features: plain, scaled
    linearly by 4, or scaled by 8 in the slow dimensions alone (fewer than 1 turn over 4096 tokens;
    more than 32 turns: unscaled; a ramp between)."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "yarn":
        at = [rot * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(10000.0)) for n in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        return f * (1.0 - ramp) + f / 8.0 * ramp, 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    c, s = dict(case), {"case": dict(case)}
    td = TYPES[c["dtype"]]
    B, T = c["B"], c["T"]
    if c["op"] == "recurrence":
        D = c["D"]
        shape = (B, T, D)
        rate = torch.exp(torch.empty((D,), device=dev).uniform_(math.log(0.01), 0.0, generator=g))  # of each channel
        log_a = -rate * torch.sigmoid(normal(*shape))
        if c["gate"] == "log":
            gate = log_a
        elif c["gate"] == "decay":
            gate = torch.exp(log_a)
        else:
            gate = log_a - torch.log(-torch.expm1(log_a))
        if c["docs"]:  # a new document's first token drops the state
            first = torch.rand((B, T, 1), generator=g, device=dev) < 1.0 / c["docs"]
            gate = torch.where(first, torch.tensor(0.0 if c["gate"] == "decay" else -math.inf, device=dev), gate)
        s["x"], s["gate"] = normal(*shape).to(td), gate.to(TYPES[c["gate_dtype"]])
        s["h0"] = normal(B, D) if c["h0"] else None
        s["lengths"] = None
        if c["ragged"]:
            s["lengths"] = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
            s["lengths"][0] = T
        if c["mode"] == "train":
            s["dh"], s["dfinal"] = normal(*shape).to(td), normal(B, D)
        if c["mode"] == "step":
            s["x"], s["gate"], s["state"] = s["x"][:, 0].contiguous(), s["gate"][:, 0].contiguous(), normal(B, D)
    else:
        Hq, Hk, W = c["Hq"], c["Hk"], c["width"]
        fused = normal(B, T, Hq + 2 * Hk, W).to(td)  # queries, keys and values of one projection
        s["q"], s["k"] = fused[:, :, :Hq], fused[:, :, Hq:Hq + Hk]
        freqs, s["amplitude"] = _frequencies(c["rot"], c["scaling"])
        s["freqs"] = freqs.to(dev)
        at = torch.randint(0, c["start"] + 1, (B, 1), generator=g, device=dev)
        s["positions"] = at + torch.arange(T, device=dev)[None]
        if c["op"] == "qk_norm":
            rms = c["norm"] == "rms"
            s["wq"] = 1.0 + 0.1 * normal(W) if rms else None
            s["wk"] = 1.0 + 0.1 * normal(W) if rms else None
            s["scale_q"] = 1.0 if rms else W ** -0.5
        if c["mode"] == "train":
            s["dq"] = normal(B, T, Hq, W).to(td)
            s["dk"] = normal(B, T, Hk, W).to(td)
    return s


def _decay(gate, kind):
    """a, 1 - a and da / dgate in the gate's precision."""
    if kind == "log":
        a = torch.exp(gate)
        return a, -torch.expm1(gate), a
    if kind == "logit":
        a, b = torch.sigmoid(gate), torch.sigmoid(-gate)
        return a, b, a * b
    return gate, 1.0 - gate, torch.ones_like(gate)


def _input_scale(a, b, kind):
    """s and ds / da."""
    if kind == "complement":
        return b, -torch.ones_like(a)
    if kind == "norm":
        s = torch.sqrt(b * (1.0 + a))
        return s, torch.where(s > 0, -a / s, torch.zeros_like(s))
    return torch.ones_like(a), torch.zeros_like(a)


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dimension 1 from 0, by doubling."""
    step = 1
    while step < a.shape[1]:
        u = torch.cat([u[:, :step], u[:, step:] + a[:, step:] * u[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return u


def _plain_recurrence(s):
    c = s["case"]
    x, gate = s["x"].float(), s["gate"].float()
    a, b, da = _decay(gate, c["gate"])
    sc, dsc = _input_scale(a, b, c["scale"])
    if c["mode"] == "step":
        s["state"].copy_(a * s["state"] + sc * x)
        return [s["state"].to(s["x"].dtype), s["state"]]
    inside = None
    if s["lengths"] is not None:
        inside = (torch.arange(c["T"], device=x.device)[None] < s["lengths"][:, None])[..., None]
        a, sc = torch.where(inside, a, 1.0), torch.where(inside, sc, 0.0)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros_like(x[:, 0])
    u = sc * x
    u[:, 0] += a[:, 0] * h0
    h = _scan(a, u)
    final = h[:, -1].clone()
    out = [(h if inside is None else torch.where(inside, h, 0.0)).to(s["x"].dtype), final]
    if c["mode"] == "train":
        lam = s["dh"].float()
        if inside is not None:
            lam = torch.where(inside, lam, 0.0)
        lam[:, -1] += s["dfinal"]
        ahead = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        lam = _scan(ahead.flip(1), lam.flip(1)).flip(1)
        before = torch.cat([h0[:, None], h[:, :-1]], 1)
        dgate = lam * da * (before + dsc * x)
        if inside is not None:
            dgate = torch.where(inside, dgate, 0.0)
        out += [(lam * sc).to(s["x"].dtype), dgate.to(s["gate"].dtype), a[:, 0] * lam[:, 0]]
    return out


def _cos_sin(s):
    angle = s["positions"].double()[..., None] * s["freqs"]
    return (torch.cos(angle) * s["amplitude"]).float()[:, :, None], (torch.sin(angle) * s["amplitude"]).float()[:, :, None]


def _rotate(y, cos, sin, rot, layout):
    if layout == "half":
        y1, y2 = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([y1 * cos - y2 * sin, y2 * cos + y1 * sin], -1)
    else:
        y1, y2 = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([y1 * cos - y2 * sin, y2 * cos + y1 * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_heads(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    out, grads = [], []
    for name, scale in (("q", s.get("scale_q", 1.0)), ("k", 1.0)):
        if name == "k" and not c["Hk"]:
            break
        x = s[name].float()
        y = x
        w = s.get("w" + name)
        if c["norm"] != "none":
            n = c["width"] if c["norm"] == "rms" else 1
            inv = torch.rsqrt((x * x).sum(-1, keepdim=True) / n + EPS)
            y = x * inv * scale
            if w is not None:
                y = y * w
        out.append(_rotate(y, cos, sin, c["rot"], c["layout"]).to(s[name].dtype))
        if c["mode"] == "train":
            g = _rotate(s["d" + name].float(), cos, -sin, c["rot"], c["layout"])
            if c["norm"] != "none":
                g = g * scale
                dw = (g * x * inv).sum((0, 1, 2)) if w is not None else None
                if w is not None:
                    g = g * w
                g = inv * (g - x * (inv * inv / n) * (g * x).sum(-1, keepdim=True))
                if dw is not None:
                    grads.append(dw)
            grads.append(g.to(s[name].dtype))
    return out + grads


def _own_recurrence(s):
    import preconditioned_delta_rule_token_b200 as pk
    c = s["case"]
    how = {"gate_form": c["gate"], "input_scale": c["scale"]}
    if c["mode"] == "step":
        return [pk.recurrence_step(s["x"], s["gate"], s["state"], **how), s["state"]]
    if c["mode"] == "forward":
        return list(pk.recurrence(s["x"], s["gate"], h0=s["h0"], lengths=s["lengths"], **how))
    h, final, marks = pk.recurrence(s["x"], s["gate"], h0=s["h0"], lengths=s["lengths"], checkpoints=True, **how)
    dfinal = s["dfinal"]
    if s["lengths"] is None and s["dh"].dtype == torch.float32:
        # the plain form adds the final state's gradient into dh in place there: the state goes the same way here
        s["dh"][:, -1] += dfinal
        dfinal = None
    g = pk.recurrence_backward(s["x"], s["gate"], s["dh"], h0=s["h0"], dfinal_h=dfinal, lengths=s["lengths"],
                               checkpoints=marks, **how)
    return [h, final, g["dx"], g["dgate"], g["dh0"]]


def _own_heads(s):
    import preconditioned_delta_rule_token_b200 as pk
    c = s["case"]
    how = {"positions": s["positions"], "layout": c["layout"], "amplitude": s["amplitude"]}
    if c["op"] == "rope":
        out = [pk.rope(s["q"], s["freqs"], **how)]
        if c["mode"] == "train":
            out.append(pk.rope(s["dq"], s["freqs"], inverse=True, **how))
        return out
    how.update(freqs=s["freqs"], norm=c["norm"], eps=EPS, wq=s["wq"], wk=s["wk"], scale_q=s["scale_q"])
    out = list(pk.qk_norm(s["q"], s["k"], **how))
    if c["mode"] == "train":
        g = pk.qk_norm_backward(s["q"], s["k"], s["dq"], s["dk"], **how)
        for name in ("q", "k"):
            if s["w" + name] is not None:
                out.append(g["dw" + name])
            out.append(g["d" + name])
    return out


def run(state):
    if state["case"]["op"] == "recurrence":
        return _own_recurrence(state) if own else _plain_recurrence(state)
    return _own_heads(state) if own else _plain_heads(state)


def work(case):
    """Each input read once, each output written once; the operations of the formulas, a function of
    one number (exp, sqrt, a quotient) counted as one."""
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "recurrence":
        n, rows = c["B"] * c["T"] * c["D"], c["B"] * c["D"]
        eg = 2 if c["gate_dtype"] == "bf16" else 4
        if c["mode"] == "step":
            return {"bytes": n * (2 * e + eg + 8), "flops": 8 * n}
        b = n * (2 * e + eg) + 4 * rows * (2 if c["h0"] else 1)
        if c["mode"] == "train":
            b += n * (2 * e + eg) + 8 * rows
        return {"bytes": b, "flops": (8 if c["mode"] == "forward" else 20) * n}
    n = c["B"] * c["T"] * (c["Hq"] + c["Hk"]) * c["width"]
    train = c["mode"] == "train"
    return {"bytes": n * e * (4 if train else 2) + 8 * c["B"] * c["T"], "flops": n * (18 if train else 7)}


def _exact_recurrence(s):
    """Token after token in 64 bits; the gradients by the reversed walk."""
    c = s["case"]
    x, gate = s["x"].double(), s["gate"].double()
    if c["gate"] == "log":
        a = gate.exp()
        one_less, slope = -torch.expm1(gate), a
    elif c["gate"] == "logit":
        a = 1.0 / (1.0 + (-gate).exp())
        one_less = 1.0 / (1.0 + gate.exp())
        slope = a * one_less
    else:
        a, one_less, slope = gate, 1.0 - gate, torch.ones_like(gate)
    scale = {"none": lambda: torch.ones_like(a), "complement": lambda: one_less,
             "norm": lambda: (one_less * (1.0 + a)).sqrt()}[c["scale"]]()
    if c["mode"] == "step":
        state = a * s["state"].double() + scale * x
        return [state, state]
    B, T, D = x.shape
    h = torch.zeros((B, D), dtype=torch.float64, device=x.device) if s["h0"] is None else s["h0"].double()
    lengths = torch.full((B,), T, device=x.device) if s["lengths"] is None else s["lengths"].long()
    live = (torch.arange(T, device=x.device)[:, None] < lengths[None])[..., None]  # [T, B, 1]
    states = torch.empty((T + 1, B, D), dtype=torch.float64, device=x.device)
    states[0] = h
    for t in range(T):
        h = torch.where(live[t], a[:, t] * h + scale[:, t] * x[:, t], h)
        states[t + 1] = h
    rows = states[1:].permute(1, 0, 2)
    mask = live.permute(1, 0, 2)
    out = [torch.where(mask, rows, 0.0), h]
    if c["mode"] == "train":
        dx, dgate = torch.zeros_like(x), torch.zeros_like(x)
        lam = s["dfinal"].double()
        for t in range(T - 1, -1, -1):
            here = lam + s["dh"][:, t].double()
            da = here * states[t]
            if c["scale"] == "complement":
                da = da - here * x[:, t]
            elif c["scale"] == "norm":
                da = da - here * x[:, t] * a[:, t] / scale[:, t]
            dx[:, t] = torch.where(live[t], here * scale[:, t], 0.0)
            dgate[:, t] = torch.where(live[t], da * slope[:, t], 0.0)
            lam = torch.where(live[t], a[:, t] * here, lam)
        out += [dx, dgate, lam]
    return out


def _exact_heads(s):
    """The rotation as complex products in 64 bits, the gradients by differentiating it."""
    c = s["case"]
    turn = torch.polar(torch.full_like(s["positions"].double()[..., None] * s["freqs"], s["amplitude"]),
                       s["positions"].double()[..., None] * s["freqs"])[:, :, None]
    out, grads = [], []
    for name in ("q", "k"):
        H = c["Hq"] if name == "q" else c["Hk"]
        if not H:
            continue
        x = s[name].double().requires_grad_(c["mode"] == "train")
        w = s.get("w" + name)
        w = w.double().requires_grad_(c["mode"] == "train") if w is not None else None
        y = x
        if c["norm"] != "none":
            power = x.square().mean(-1, keepdim=True) if c["norm"] == "rms" else x.square().sum(-1, keepdim=True)
            y = x / (power + EPS).sqrt()
            y = y * w if w is not None else y
            y = y * (s["scale_q"] if name == "q" else 1.0)
        head = y[..., :c["rot"]].unflatten(-1, (2, -1) if c["layout"] == "half" else (-1, 2))
        pair = -2 if c["layout"] == "half" else -1
        z = torch.complex(head.select(pair, 0), head.select(pair, 1)) * turn
        z = torch.stack([z.real, z.imag], pair).flatten(-2)
        y = torch.cat([z, y[..., c["rot"]:]], -1)
        out.append(y.detach())
        if c["mode"] == "train":
            got = torch.autograd.grad(y, [x] if w is None else [w, x], s["d" + name].double())
            grads += list(got)
    return out + grads


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_recurrence(s) if case["op"] == "recurrence" else _exact_heads(s)
