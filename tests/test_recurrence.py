"""The gated linear recurrence: forward, backward, single-token step.

    h_t = a_t h_{t-1} + s_t x_t, a from the gate (decay, log, logit), s = 1, 1 - a or sqrt(1 - a^2).

Tolerances, fixed before the first run. One token costs the fp32 evaluation at most 12 roundings of the
terms it carries (the gate's function 8: an exponential and a quotient within 2 units in the last place each
and a sum; the product, the sum and the joining of the runs 4), and a term is carried over at most T tokens;
the last terms themselves carry s and its products, 48 more. So an output lies within
(12 T + 48) 2^-24 of the walk over absolute values, plus half a step of its own type; dgate multiplies two
such walks, 24 T + 96."""
import ctypes

import pytest
import torch

from tests import _layer_ref as ref

FORMS, SCALES = ("decay", "log", "logit"), ("none", "complement", "norm")
TYPES = ((torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32))
SHAPES = ((1, 1, 1), (2, 7, 5), (1, 63, 32), (2, 64, 130), (3, 65, 128), (2, 200, 36), (1, 300, 258), (5, 17, 512))


def case(seed, B, T, D, dt, gdt, form, resets=True):
    g = torch.Generator().manual_seed(seed)
    x, dh = torch.randn(B, T, D, generator=g).to(dt), torch.randn(B, T, D, generator=g).to(dt)
    log_a = -torch.exp(torch.empty(B, T, D).uniform_(-6.0, 1.0, generator=g))
    gate = {"decay": log_a.exp(), "log": log_a, "logit": log_a - torch.log(-torch.expm1(log_a))}[form]
    if resets:
        gate[torch.rand(B, T, generator=g) < 0.05] = 0.0 if form == "decay" else -float("inf")
    h0, dfinal = torch.randn(B, D, generator=g), torch.randn(B, D, generator=g)
    return x, gate.to(gdt), dh, h0, dfinal


# ------------------------------------------------------------------ CPU: the formulas and the refusals

@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scale", SCALES)
def test_the_gradient_formulas_agree_with_differences(form, scale):
    """Central differences of the float64 walk, for every input."""
    x, gate, dh, h0, dfinal = (t.double() for t in case(3, 2, 6, 3, torch.float32, torch.float32, form, resets=False))
    lengths = torch.tensor([6, 4])
    inside = (torch.arange(6)[None] < lengths[:, None])[..., None]

    def loss(x, gate, h0):
        h, f, _, _ = ref.recurrence(x, gate, h0, lengths, form, scale)
        return float((h * dh * inside).sum() + (f * dfinal).sum())

    got = ref.recurrence_grads(x, gate, dh, h0, dfinal, lengths, form, scale)
    for name, k in (("dx", 0), ("dgate", 1), ("dh0", 2)):
        args = [x, gate, h0]
        for i in range(args[k].numel()):
            e = torch.zeros(args[k].numel(), dtype=torch.float64)
            e[i] = 1e-6
            e = e.view_as(args[k])
            diff = (loss(*[a + e if j == k else a for j, a in enumerate(args)]) -
                    loss(*[a - e if j == k else a for j, a in enumerate(args)])) / 2e-6
            assert abs(diff - float(got[name][0].flatten()[i])) < 1e-6 * (1 + abs(diff)), (name, i)


def _params(lib_, **kw):
    p = lib_.osdn_recur_params()
    p.struct_size = ctypes.sizeof(p)
    a = dict(B=2, T=100, D=48, dtype=0, gate_dtype=0, gate_form=0, input_scale=0)
    a.update(kw)
    for k, v in a.items():
        if k.startswith("stride"):
            getattr(p, k)[:] = v
        else:
            setattr(p, k, v)
    return p


def test_arguments_are_checked_on_the_host(osdn_lib):
    B, L = osdn_lib, osdn_lib.lib()
    n = ctypes.c_size_t(0)
    assert ctypes.sizeof(B.osdn_recur_params) == 88
    assert L.osdn_recur_bwd_workspace_size(_params(B), ctypes.byref(n)) == 0 and n.value >= 2 * 2 * 48 * 4
    inv, uns = B.OSDN_ERR_INVALID_ARG, B.OSDN_ERR_UNSUPPORTED
    for kw, code in ((dict(B=0), inv), (dict(T=-1), inv), (dict(D=0), inv), (dict(D=1 << 25), inv), (dict(dtype=2), inv),
                     (dict(gate_dtype=7), inv), (dict(dtype=1, gate_dtype=0), uns), (dict(gate_form=3), inv),
                     (dict(input_scale=-1), inv), (dict(stride_x=(-8, 48)), inv), (dict(stride_h=(1 << 39, 48)), inv),
                     (dict(T=(1 << 30) + 1), inv), (dict(reserved=1), inv), (dict(B=1 << 30, D=1 << 20, T=1), inv)):
        assert L.osdn_recur_bwd_workspace_size(_params(B, **kw), ctypes.byref(n)) == code, kw
        assert B.get_last_error()
    p = _params(B)
    p.struct_size = 40
    assert L.osdn_recur_bwd_workspace_size(p, ctypes.byref(n)) == inv
    assert L.osdn_recur_bwd_workspace_size(_params(B), None) == inv
    assert L.osdn_recur_bwd_workspace_size(None, ctypes.byref(n)) == inv


def test_pointers_are_checked_on_the_host(osdn_lib):
    B, L = osdn_lib, osdn_lib.lib()
    inv = B.OSDN_ERR_INVALID_ARG
    f = [(1 << 20) + (i << 16) for i in range(12)]    # never dereferenced: the checks fail first
    odd = (1 << 20) + 1
    assert L.osdn_recur_fwd(_params(B), None, f[1], None, None, f[2], None, None, None) == inv
    assert "NULL" in B.get_last_error()
    assert L.osdn_recur_fwd(_params(B), f[0], odd, None, None, f[2], None, None, None) == inv
    assert L.osdn_recur_fwd(_params(B), f[0], f[1], (1 << 20) + 4, None, f[2], None, None, None) == inv
    assert L.osdn_recur_fwd(_params(B), f[0], f[1], None, None, f[0], None, None, None) == inv
    assert L.osdn_recur_fwd(_params(B, stride_h=(48, 48)), f[0], f[1], None, None, f[2], None, None, None) == inv
    assert "overlap" in B.get_last_error()
    bwd = lambda **kw: L.osdn_recur_bwd(  # noqa: E731
        _params(B), *[kw.get(n, d) for n, d in (("x", f[0]), ("gate", f[1]), ("h0", None), ("lengths", None),
                                               ("dh", f[2]), ("dfinal", None), ("marks", f[3]), ("dx", f[4]),
                                               ("dgate", f[5]), ("dh0", None), ("ws", None), ("bytes", 0),
                                               ("stream", None))])
    for kw in (dict(x=None), dict(dh=None), dict(dx=None), dict(dgate=None), dict(dx=f[0]), dict(dgate=f[2]),
               dict(dx=f[5]), dict(marks=None), dict(marks=None, ws=f[6], bytes=16), dict(dx=f[4] + 4)):
        assert bwd(**kw) == inv, kw
    assert L.osdn_recur_step(_params(B), f[0], f[1], None, f[2], None) == inv
    assert L.osdn_recur_step(_params(B), f[0], f[1], f[3], f[0], None) == inv


def test_the_wrappers_refuse_what_they_cannot_take():
    import preconditioned_delta_rule_token_b200 as pk
    x = torch.zeros(2, 4, 8)
    for call in (lambda: pk.recurrence(x, x), lambda: pk.recurrence_backward(x, x, x),
                 lambda: pk.recurrence_step(x[:, 0], x[:, 0], torch.zeros(2, 8)), lambda: pk.recurrence(x[0], x[0])):
        with pytest.raises(pk.OsdnError):
            call()


# ------------------------------------------------------------------ GPU

def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _check_all(B, T, D, dt, gdt, form, scale, seed=1, lengths=None, with_state=True):
    import preconditioned_delta_rule_token_b200 as pk
    x, gate, dh, h0, dfinal = case(seed, B, T, D, dt, gdt, form)
    if not with_state:
        h0 = dfinal = None
    xs, gs, ds, hs, fs, ns = _cuda(x, gate, dh, h0, dfinal, lengths)
    how = dict(lengths=ns, gate_form=form, input_scale=scale)
    h, final, marks = pk.recurrence(xs, gs, h0=hs, checkpoints=True, **how)
    want_h, want_f, mh, mf = ref.recurrence(x, gate, h0, lengths, form, scale)
    ref.close(h, want_h, mh, 12 * T + 48, "h")
    ref.close(final, want_f, mf, 12 * T + 48, "final")
    g = pk.recurrence_backward(xs, gs, ds, h0=hs, dfinal_h=fs, checkpoints=marks, **how)
    want = ref.recurrence_grads(x, gate, dh, h0, dfinal, lengths, form, scale)
    ref.close(g["dx"], *want["dx"], 12 * T + 48, "dx")
    ref.close(g["dh0"], *want["dh0"], 12 * T + 48, "dh0")
    ref.close(g["dgate"], *want["dgate"], 24 * T + 96, "dgate")
    again = pk.recurrence_backward(xs, gs, ds, h0=hs, dfinal_h=fs, **how)   # without the saved states
    assert all(torch.equal(g[k], again[k]) for k in g)
    assert pk.osdn_sync_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("types", TYPES)
def test_forward_and_backward_over_shapes(shape, types):
    _check_all(*shape, *types, "log", "complement")


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("types", TYPES)
def test_forward_and_backward_over_gates(form, scale, types):
    _check_all(2, 77, 40, *types, form, scale, seed=2, with_state=form != "log")


@pytest.mark.gpu
@pytest.mark.parametrize("D", (24, 33))
def test_lengths_leave_later_rows_alone(D):
    """Lengths of 0, 1, a tile, T and beyond T (taken as T); a negative one is 0."""
    import preconditioned_delta_rule_token_b200 as pk
    lengths = torch.tensor([0, 1, 64, 65, 130, 500, -3], dtype=torch.int32)
    _check_all(7, 130, D, torch.float32, torch.float32, "logit", "norm", seed=4, lengths=lengths)
    x, gate, dh, h0, _ = case(4, 7, 130, D, torch.bfloat16, torch.bfloat16, "decay")
    n = [min(max(int(v), 0), 130) for v in lengths]
    for b in range(7):   # what lies behind a length is not read
        x[b, n[b]:] = gate[b, n[b]:] = dh[b, n[b]:] = float("nan")
    xs, gs, ds, hs, ns = _cuda(x, gate, dh, h0, lengths)
    h = torch.full_like(xs, 7.0)
    _, final = pk.recurrence(xs, gs, h0=hs, lengths=ns, h=h)
    g = pk.recurrence_backward(xs, gs, ds, h0=hs, lengths=ns)
    assert torch.isfinite(final).all() and torch.equal(final[0], hs[0]) and torch.equal(final[6], hs[6])
    for b in range(7):
        assert bool((h[b, n[b]:] == 7.0).all()) and bool(torch.isfinite(h[b]).all())
        assert bool(torch.isfinite(g["dx"][b]).all()) and bool((g["dgate"][b, n[b]:] == 0).all())
        assert bool((g["dx"][b, n[b]:] == 0).all())
    own = pk.recurrence(xs, gs, h0=hs, lengths=ns)[0]   # without h: zeros there
    assert all(bool((own[b, n[b]:] == 0).all()) and torch.equal(own[b, :n[b]], h[b, :n[b]]) for b in range(7))


@pytest.mark.gpu
@pytest.mark.parametrize("T", (1000, 4133))
@pytest.mark.parametrize("D", (32, 200, 1030))
def test_long_sequences(T, D):
    """Few channels: the work is split over the tokens."""
    _check_all(1, T, D, torch.bfloat16, torch.float32, "log", "none", seed=5)


@pytest.mark.gpu
def test_many_sequences():
    _check_all(64, 70, 512, torch.bfloat16, torch.bfloat16, "logit", "complement", seed=6)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", (0, 8, 2, 1))
def test_column_slices_and_other_orders(offset):
    """x, gate and h as column slices of wider buffers, at every alignment, and time-major tensors: the
    same values as dense tensors, and the columns between them untouched."""
    import preconditioned_delta_rule_token_b200 as pk
    B, T, D = 2, 150, 40
    x, gate, dh, h0, dfinal = case(8, B, T, D, torch.bfloat16, torch.bfloat16, "logit")
    W = 3 * D + 16
    buf = torch.full((B, T, W), 5.0, dtype=torch.bfloat16, device="cuda")
    xs, gs, hs = (buf[..., offset + i * D:offset + (i + 1) * D] for i in range(3))
    xs.copy_(x), gs.copy_(gate)
    want = pk.recurrence(x.cuda(), gate.cuda(), h0=h0.cuda(), gate_form="logit", checkpoints=True)
    got = pk.recurrence(xs, gs, h0=h0.cuda(), gate_form="logit", h=hs, checkpoints=True)
    ref.close(got[0], f := ref.f64(want[0]), f.abs(), 4 * 2 ** 16, "h")   # within a step of bf16
    ref.close(got[1], f := ref.f64(want[1]), f.abs(), 12 * T + 48, "final")
    edge = torch.cat([buf[..., :offset], buf[..., offset + 3 * D:]], -1)
    assert bool((edge == 5.0).all())
    tm = [t.cuda().transpose(0, 1).contiguous().transpose(0, 1) for t in (x, gate, dh)]   # time-major memory
    got = pk.recurrence(tm[0], tm[1], h0=h0.cuda(), gate_form="logit", checkpoints=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    a = pk.recurrence_backward(*tm, h0=h0.cuda(), dfinal_h=dfinal.cuda(), gate_form="logit")
    b = pk.recurrence_backward(x.cuda(), gate.cuda(), dh.cuda(), h0=h0.cuda(), dfinal_h=dfinal.cuda(), gate_form="logit")
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.gpu
def test_one_gate_for_the_batch():
    """A gate expanded over the sequences (stride 0) equals the gate in memory."""
    import preconditioned_delta_rule_token_b200 as pk
    x, gate, _, _, _ = case(9, 4, 90, 64, torch.float32, torch.float32, "decay")
    one = gate[:1].cuda()
    assert torch.equal(pk.recurrence(x.cuda(), one.expand(4, -1, -1))[0],
                       pk.recurrence(x.cuda(), one.expand(4, -1, -1).contiguous())[0])
    with pytest.raises(pk.OsdnError):
        pk.recurrence(x.cuda(), one[:, :1].expand(4, 90, -1))
    dh = torch.randn(4, 90, 64, generator=torch.Generator().manual_seed(1)).cuda()
    a = pk.recurrence_backward(x.cuda(), one.expand(4, -1, -1), dh[:1].expand(4, -1, -1))
    b = pk.recurrence_backward(x.cuda(), one.expand(4, -1, -1).contiguous(), dh[:1].expand(4, -1, -1).contiguous())
    assert all(torch.equal(a[k], b[k]) for k in a) and a["dgate"].shape == (4, 90, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,dt", ((1, 1, 5000, torch.bfloat16), (300, 3, 8, torch.float32), (1, 2049, 72, torch.float32)))
def test_corners_of_the_grid(B, T, D, dt):
    """One token, more sequences than SMs with a handful of channels, one token past 16 tiles of 128."""
    _check_all(B, T, D, dt, torch.float32, "decay", "complement", seed=21)


@pytest.mark.gpu
def test_no_tokens():
    import preconditioned_delta_rule_token_b200 as pk
    x, h0 = torch.zeros(2, 0, 8, device="cuda"), torch.randn(2, 8, device="cuda")
    h, final, marks = pk.recurrence(x, x, h0=h0, checkpoints=True)
    assert h.shape == (2, 0, 8) and marks.shape == (2, 0, 8) and torch.equal(final, h0)
    g = pk.recurrence_backward(x, x, x, h0=h0, dfinal_h=h0)
    assert torch.equal(g["dh0"], h0) and g["dx"].numel() == 0
    assert bool((pk.recurrence(x, x)[1] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", (1, 30, 64, 1030))
def test_steps_continue_a_forward(types, D):
    """Single tokens from a forward's final state, against the walk over all tokens."""
    import preconditioned_delta_rule_token_b200 as pk
    x, gate, _, h0, _ = case(11, 3, 20, D, *types, "logit")
    xs, gs, hs = _cuda(x, gate, h0)
    how = dict(gate_form="logit", input_scale="norm")
    _, state = pk.recurrence(xs[:, :12].contiguous(), gs[:, :12].contiguous(), h0=hs, **how)
    outs = [pk.recurrence_step(xs[:, t], gs[:, t], state, **how) for t in range(12, 20)]
    want_h, want_f, mh, mf = ref.recurrence(x, gate, h0, None, "logit", "norm")
    ref.close(torch.stack(outs, 1), want_h[:, 12:], mh[:, 12:], 12 * 20 + 48, "steps")
    ref.close(state, want_f, mf, 12 * 20 + 48, "state")


@pytest.mark.gpu
def test_gates_at_the_edges():
    """Gates of exactly 1 and 0, of the type's lowest value and of both infinities stay finite, forward and
    backward; a gate of -inf (a = 0) makes every later state independent of what came before."""
    import preconditioned_delta_rule_token_b200 as pk
    low = torch.finfo(torch.bfloat16).min
    for form, values in (("decay", (0.0, 1.0)), ("log", (-float("inf"), low, 0.0, -1e-30)),
                         ("logit", (-float("inf"), float("inf"), low, -low, 0.0))):
        for scale in SCALES:
            x, _, dh, h0, dfinal = case(12, 2, 66, 32, torch.bfloat16, torch.bfloat16, form)
            g = torch.Generator().manual_seed(1)
            gate = torch.tensor(values)[torch.randint(0, len(values), (2, 66, 32), generator=g)].to(torch.bfloat16)
            h, f = pk.recurrence(x.cuda(), gate.cuda(), h0=h0.cuda(), gate_form=form, input_scale=scale)
            want_h, want_f, mh, mf = ref.recurrence(x, gate, h0, None, form, scale)
            ref.close(h, want_h, mh, 12 * 66 + 48, (form, scale))
            ref.close(f, want_f, mf, 12 * 66 + 48, (form, scale))
            got = pk.recurrence_backward(x.cuda(), gate.cuda(), dh.cuda(), h0=h0.cuda(), dfinal_h=dfinal.cuda(),
                                         gate_form=form, input_scale=scale)
            want = ref.recurrence_grads(x, gate, dh, h0, dfinal, None, form, scale)
            for k in got:
                ref.close(got[k], *want[k], 24 * 66 + 96, (form, scale, k))


@pytest.mark.gpu
def test_against_differences_on_the_device():
    """A directional derivative of the fp32 forward. The difference quotient over 2 eps = 2^-5 is off by at
    most eps^2 of third derivatives (the loss is linear in x and h0; in the gate its terms are bounded
    by their magnitude) and by the forward's rounding over 2 eps: within 1e-2 of the magnitude sum."""
    import preconditioned_delta_rule_token_b200 as pk
    x, gate, dh, h0, dfinal = _cuda(*case(13, 2, 40, 64, torch.float32, torch.float32, "log", resets=False))
    g = torch.Generator(device="cuda").manual_seed(2)
    how = dict(gate_form="log", input_scale="complement")
    got = pk.recurrence_backward(x, gate, dh, h0=h0, dfinal_h=dfinal, **how)
    for name, base in (("dx", x), ("dgate", gate), ("dh0", h0)):
        v = torch.randn(base.shape, generator=g, device="cuda") * (base.abs() if name == "dgate" else 1.0)

        def loss(e):
            h, f = pk.recurrence(x + e * v if name == "dx" else x, gate + e * v if name == "dgate" else gate,
                                 h0=h0 + e * v if name == "dh0" else h0, **how)
            return float((h.double() * dh).sum() + (f.double() * dfinal).sum())

        eps = 2.0 ** -6
        diff, want = (loss(eps) - loss(-eps)) / (2 * eps), got[name].double() * v
        assert abs(diff - float(want.sum())) <= 1e-2 * float(want.abs().sum()), name


@pytest.mark.gpu
def test_repeats_other_streams_and_graphs():
    """Bitwise the same from call to call, on a side stream, and replayed from a graph with new inputs."""
    import preconditioned_delta_rule_token_b200 as pk
    how = dict(gate_form="logit", input_scale="complement")
    x, gate, dh, h0, dfinal = _cuda(*case(14, 2, 700, 72, torch.bfloat16, torch.bfloat16, "logit"))
    x2 = torch.randn(2, 700, 72, device="cuda").bfloat16()

    def run(x, stream=None):
        h, f, marks = pk.recurrence(x, gate, h0=h0, checkpoints=True, stream=stream, **how)
        g = pk.recurrence_backward(x, gate, dh, h0=h0, dfinal_h=dfinal, checkpoints=marks, stream=stream, **how)
        return [h, f, g["dx"], g["dgate"], g["dh0"]]

    want, want2 = run(x), run(x2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    static = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(static)
    for src, exp in ((x2, want2), (x, want)):
        static.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(exp, out))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows 2^30 elements apart: the third lies past 2^31."""
    import preconditioned_delta_rule_token_b200 as pk
    D, step = 40, 1 << 30
    buf = torch.zeros(2 * step + 256, dtype=torch.bfloat16, device="cuda")
    view = lambda off: torch.as_strided(buf, (1, 3, D), (0, step, 1), off)  # noqa: E731
    x, gate, dh, h0, _ = case(15, 1, 3, D, torch.bfloat16, torch.bfloat16, "decay")
    xs, gs, hs, ds = view(0), view(48), view(96), view(144)
    xs.copy_(x), gs.copy_(gate), ds.copy_(dh)
    _, f = pk.recurrence(xs, gs, h0=h0.cuda(), h=hs)
    want = pk.recurrence(x.cuda(), gate.cuda(), h0=h0.cuda())
    assert torch.equal(hs, want[0]) and torch.equal(f, want[1])
    a = pk.recurrence_backward(xs, gs, ds, h0=h0.cuda())
    b = pk.recurrence_backward(x.cuda(), gate.cuda(), dh.cuda(), h0=h0.cuda())
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D", ((1, 1500, 64), (40, 300, 512), (1, 32768, 1024), (32, 512, 2048)))
def test_a_wait_that_gives_up_is_reported(B, T, D):
    """With waits bounded to 1 ns those for memory give up (alone and in a cluster): the call ends, the status
    says so, and the next call is right again."""
    import preconditioned_delta_rule_token_b200 as pk
    x, gate, dh = (torch.randn(B, T, D, device="cuda").bfloat16() for _ in range(3))
    want = pk.recurrence(x, gate, gate_form="logit", checkpoints=True)
    grads = pk.recurrence_backward(x, gate, dh, checkpoints=want[2], gate_form="logit")
    assert pk.osdn_sync_status() == pk.OSDN_OK
    for call in (lambda: pk.recurrence(x, gate, gate_form="logit"),
                 lambda: pk.recurrence_backward(x, gate, dh, checkpoints=want[2], gate_form="logit")):
        pk.osdn_set_wait_limit_ns(1)
        try:
            call()
            status = pk.osdn_sync_status()
        finally:
            pk.osdn_set_wait_limit_ns(0)
        assert status == pk.OSDN_ERR_TIMEOUT and pk.osdn_sync_status() == pk.OSDN_OK
    got = pk.recurrence(x, gate, gate_form="logit", checkpoints=True)
    again = pk.recurrence_backward(x, gate, dh, checkpoints=got[2], gate_form="logit")
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and all(torch.equal(grads[k], again[k]) for k in grads)
    assert pk.osdn_sync_status() == pk.OSDN_OK
